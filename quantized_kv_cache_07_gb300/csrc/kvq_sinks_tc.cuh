// Chunked prefill with sinks and a sliding window on tcgen05 (kvq_prefill_sinks, KVQ_PREFILL_UNITS).
//
// A unit is up to 256 query vectors: 256 / G consecutive rows of the call x the G query heads of one KV head.  A
// CTA takes units in turn and, for every sequence among a unit's rows (a "pass", mostly one), streams the tiles of
// 64 tokens of the sinks, then from the shortest row's window to the longest row's end.  The products, the
// softmax and the conversion of codes are those of kvq_shared_tc.cu, which has the layouts and the roles:
//   warpgroups 0 and 1 softmax, warpgroup 2 converts, warps 12 and 14 issue the products of one softmax warpgroup each,
// and warp 13 plans: it reads the rows of the next unit (their sequences and lengths) while this one runs.
//
// Few units: a cluster of 2, 4 or 8 CTAs takes each, every one an equal share of a pass's tiles, and they join their
// states through the cluster's shared memory (the ring's place, once the pass has drained it), each writing its share of the
// vectors.
//
// Scores.  Queries of ordinary size are scaled by one power of two, so that what turns a code product into an exponent is
// the token's alone: the converting warps store its key scale times log2(e) / sqrt(D) times that power, and an exponent
// is one fused product and sum, S s_k - (m - sigma); rows of other sizes are brought to it first.
//
// A softmax thread holds four rows of its warp's 32 and two columns of every eight, so that a scale it reads serves four
// scores: with a row a thread, each warp read all of a tile's scales for every lane, and shared memory answered 2660 requests
// of 128 bytes a tile (1024 of them operands of the products) in 2300 cycles; now 1830 in 2130.  The scales are asked for
// before the scores are waited for.
//
// Measured: 2048 rows of 32 / 8 heads on windows of 4096 (256 units of 66 tiles, int8): 171 us a call (184 with a row a
// thread), where the products alone would take 72 on all SMs; 752 on 16-vector tiles.  A tile of 256 vectors takes 2130 cycles: 1024
// of the tensor core's, whose operands also fill shared memory's port for as long, and about 1350 issued instructions a
// scheduler, which two softmax warps and a converting one do not overlap better.  A unit's start and end take 25,000 cycles,
// and 256 units are two rounds of 152 SMs.  Tried and slower: scores of the next tile while one S buffer's are at work and
// weights apart from them (198 us); queries in tensor memory, which halves the operands read, with the weights in S's only place
// (197: the products then wait for the softmax and it for them); no maximum until a sum passes its bound (255, too many
// tiles twice).  One warp that issued both warpgroups' products was itself what they waited for (195 before 187).
//
// Masks.  Row of length L sees token i < L if i < sinks or i >= L - span.  Tiles are aligned to 64 tokens; a
// tile that every row of a warp sees whole skips the mask, so it costs the tiles at the window's start and at the chunk itself.
// Blocks that no row sees are not read (their table entries may be gone): those before the shortest row's window, and
// those between the windows of rows that are further apart than a window, which are found row by row.  Of blocks that are
// read, hidden tokens have no say: scores -inf, value scales by row (as sequences stand apart in kvq_shared_tc.cu).
#pragma once

#include "kvq_tc_tiles.cuh"

namespace kvq {
namespace {

constexpr int kPlanRows = 2 * kQ;  // G = 1

struct Pass {
  int seq, least, most;  // shortest and longest row
  int far;  // rows that are not within a window of the row before: with the first alone, no token between the rows is unseen
};

struct Plan {
  int passes, h, r0, nrows;
  Pass pass[kPlanRows];
  int seq[kPlanRows], len[kPlanRows];  // by row; an empty one has sequence -1
};

struct UnitSmem {
  alignas(1024) uint8_t q[2][2][kQ * 128];  // [warpgroup][half]
  alignas(1024) TcStage st[kRing];
  float sk[kRing][kTok], sv[kRing][kTok], mk[kRing][kTok], mv[kRing][kTok];
  float svmax[kRing][4];
  float qs[2 * kQ], qz[2 * kQ];  // after a pass of one half: the second warpgroup's m and l
  int qlen[2 * kQ];
  float rm[2 * kQ], rl[2 * kQ];  // each row's m and sigma, which few tiles move; then a share's m and l, for the cluster
  // full: a stage's 128 converting threads; empty: its products are done, of both warpgroups; q_full: the softmax threads have staged a
  // pass's queries; s_full, p_full, o_done [warpgroup][S buffer]: scores, weights, P . V done; plan_full, plan_empty
  // [plan buffer]; meet: both softmax warpgroups; gather, release: the cluster's softmax threads have left their states, and
  // have read them
  uint64_t full[kRing], empty[kRing], q_full, meet, s_full[2][2], p_full[2][2], o_done[2][2], plan_full[2], plan_empty[2],
      gather, release;
  uint32_t tmem;
  Plan plan[2];
};

// A pass, walked alike by every role: tile i of this CTA's share is the pass's tile i + first, which is the sequence's,
// or that + skip from `front` on.
struct Walk {
  int seq, h, nt, first, front, skip;
  int from, most;  // no row sees the tokens between the sinks and `from`, nor those from `most` on
  bool apart;  // nor, perhaps, tokens between these: rows further apart than a window
  int nv;
  bool both;  // more than 128 vectors: both warpgroups meet every tile
  __device__ __forceinline__ int tile(int i) const { return first + i + (first + i < front ? 0 : skip); }
};
__device__ __forceinline__ Walk walk_of(const DecodeArgs& a, const Plan& p, int i, int part, int parts) {
  Walk w;
  const Pass ps = p.pass[i];
  const int all = (ps.most + kTok - 1) / kTok;
  w.seq = ps.seq;
  w.h = p.h;
  w.most = ps.most;
  w.from = max(ps.least - a.span, 0);
  w.apart = ps.far > 1;
  w.front = (min(a.sinks, ps.most) + kTok - 1) / kTok;
  w.skip = max(w.from / kTok - w.front, 0);
  const long long tiles = all - w.skip;
  w.first = int(tiles * part / parts);
  w.nt = int(tiles * (part + 1) / parts) - w.first;
  w.nv = p.nrows * a.G;
  w.both = w.nv > kQ;
  return w;
}
// Which tokens of block blk one row at least of the pass sees, as bits.
__device__ __forceinline__ uint32_t seen_tokens(const Plan& p, int seq, int blk, int sinks, int span) {
  auto below = [&](int n) { return (1u << min(max(n - blk * kBlock, 0), kBlock)) - 1u; };  // those before position n
  uint32_t m = 0;
  for (int i = 0; i < p.nrows && m != 0xFFFFu; ++i)
    if (p.seq[i] == seq) m |= below(p.len[i]) & (below(sinks) | ~below(max(p.len[i] - span, 0)));
  return m;
}
// Tiles of a pass that warpgroup j takes.
__device__ __forceinline__ int jobs_of(const Walk& g, int j) { return g.both ? g.nt : (g.nt + 1 - j) / 2; }

// The rows of unit u by one warp (`report`: errors and rows without tokens are this CTA's to deal with).
__device__ __forceinline__ void plan_unit(const DecodeArgs& a, Plan* p, int u, int rows_per, bool report, int lane) {
  const int H = a.c.H, h = u % H, r0 = (u / H) * rows_per, nrows = min(rows_per, a.B - r0);
  int passes = 0;
  for (int base = 0; base < nrows; base += 32) {
    const int i = base + lane;
    int seq = -1, len = 0;
    if (i < nrows) {
      seq = a.seq_of[r0 + i];
      if (seq < 0 || seq >= a.nseq) {
        if (h == 0 && report) flag(a.err, KVQ_DEVERR_POSITION);
        seq = -1;
      } else {
        const int most = table_tokens(a.mbps, 0);
        len = row_tokens(a.pos[r0 + i]);
        if (len < 0 || len > most) {
          if (h == 0 && report) flag(a.err, KVQ_DEVERR_SEQ_LEN);
          len = len < 0 ? 0 : most;
        }
        if (len == 0) seq = -1;
      }
      p->seq[i] = seq;
      p->len[i] = len;
    }
    __syncwarp();
    const bool near = i > 0 && i < nrows && p->seq[i - 1] == seq && abs(len - p->len[i - 1]) <= a.span;
    const uint32_t far = __ballot_sync(kFull, !near);
    uint32_t left = __ballot_sync(kFull, seq >= 0);
    while (left) {  // the sequences among these 32 rows
      const int s = __shfl_sync(kFull, seq, __ffs(left) - 1);
      const uint32_t who = __ballot_sync(kFull, seq == s);
      const int least = __reduce_min_sync(kFull, seq == s ? len : 0x7fffffff);
      const int most = __reduce_max_sync(kFull, seq == s ? len : 0);
      int at = -1;
      for (int k = 0; k < passes; k += 32) {
        const uint32_t hit = __ballot_sync(kFull, k + lane < passes && p->pass[k + lane].seq == s);
        if (hit) {
          at = k + __ffs(hit) - 1;
          break;
        }
      }
      if (lane == 0) {
        Pass& ps = p->pass[at < 0 ? passes : at];
        const int n = __popc(who & far);
        ps = at < 0 ? Pass{s, least, most, n} : Pass{s, min(ps.least, least), max(ps.most, most), ps.far + n};
      }
      passes += at < 0;
      left &= ~who;
      __syncwarp();
    }
    // rows that attend to nothing
    for (uint32_t none = report ? __ballot_sync(kFull, i < nrows && seq < 0) : 0u; none; none &= none - 1) {
      const size_t row = size_t(r0 + base + __ffs(none) - 1) * a.Hq + h * a.G;
      for (int e = lane; e < a.G * kHeadDim; e += 32) {
        if (a.out_fp32) reinterpret_cast<float*>(a.out)[row * kHeadDim + e] = 0.f;
        else reinterpret_cast<__nv_bfloat16*>(a.out)[row * kHeadDim + e] = __float2bfloat16_rn(0.f);
      }
      if (a.lse && lane < a.G) a.lse[row + lane] = kNegInf;
    }
  }
  if (lane == 0) {
    p->passes = passes;
    p->h = h;
    p->r0 = r0;
    p->nrows = nrows;
  }
}

// What a code product times its key scale is multiplied by for queries scaled by 2^kFixedExp: log2(e) / sqrt(D) / 2^kFixedExp.
constexpr float kUnitScale = kLog2e * kInvSqrtD / float(1 << kFixedExp);

constexpr uint32_t kAbs2 = 0x7FFF7FFFu;     // two bf16 values without their signs: they order as their bits
constexpr uint32_t kLeastBits = 0x3780u, kMostBits = 0x437Au;  // kFixedLeast, kFixedMost in bf16

// put_query's work for a vector of ordinary size and no factor; its sum as the product sees it (ASYM).
template <bool ASYM>
__device__ __forceinline__ float put_plain(const uint4 (&raw)[2], uint8_t* half, int row, int sub) {
  const int t = sub >> 1;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      y[k] = pack_half2(__uint_as_float(w[k] << 16) * float(1 << kFixedExp),
                        __uint_as_float(w[k] & 0xFFFF0000u) * float(1 << kFixedExp));
      if constexpr (ASYM) {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&y[k]));
        sum += h.x + h.y;
      }
    }
    *reinterpret_cast<uint4*>(half + row * 128 + ((dim_chunk(t, i) ^ (row & 7)) * 16)) = make_uint4(y[0], y[1], y[2], y[3]);
  }
  if constexpr (ASYM) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
  return sum;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 2^n, 0 below float32's normal numbers, infinity at 128.
__device__ __forceinline__ float pow2(int n) { return n < -126 ? 0.f : __uint_as_float(uint32_t(n + 127) << 23); }

// 64 columns of 16 of this warp's lanes as fragments: thread (g, t) = (lane / 4, lane % 4) holds columns 8 n + 2 t and the
// next of lanes g and g + 8; and 32 columns of packed pairs, 4 n + t, back.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16x128(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Four outputs of a row.
__device__ __forceinline__ void put_out(const DecodeArgs& a, size_t at, float4 o) {
  if (a.out_fp32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = o;
  } else {
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at) =
        make_uint2(pack_bf162(o.x, o.y), pack_bf162(o.z, o.w));
  }
}

// ---- the cluster that shares a unit
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ void remote_arrive(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote(bar, rank)) : "memory");
}
// A wait for arrivals of the cluster, whose writes are seen behind it; bounded as mbar_wait.
__device__ __forceinline__ bool cluster_wait(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}
__device__ __forceinline__ float remote_float(const void* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 remote_float4(const void* p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(remote(p, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// TWO: queries as an fp16 high and low part, the low ones in the second query tile; units of 128 vectors.
// SHARED: a cluster takes each unit (its own kernel: the join's code cost the others 7 %).
template <int KB, int VB, bool ASYM, bool TWO, bool SHARED>
__global__ void __launch_bounds__(kTcThreads, 1) sinks_tc_kernel(const DecodeArgs a, int units, int rows_per) {
  using F = Fmt<KB, VB, ASYM>;
  constexpr int kStep = kTok / kBlock;
  constexpr float kKC = KB == 8 ? 128.f : (KB == 4 ? 8.f : 2.f), kVC = VB == 8 ? 128.f : (VB == 4 ? 8.f : 2.f);
  extern __shared__ uint8_t raw_smem[];
  UnitSmem* sm = reinterpret_cast<UnitSmem*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm->full[i], 128);
      mbar_init(&sm->empty[i], 2);
    }
    mbar_init(&sm->q_full, 2 * kQ);
    mbar_init(&sm->meet, 2 * kQ);
    mbar_init(&sm->gather, 2 * kQ * cluster_size());
    mbar_init(&sm->release, 2 * kQ * cluster_size());
    for (int j = 0; j < 2; ++j) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm->s_full[j][i], 1);
        mbar_init(&sm->p_full[j][i], kQ);
        mbar_init(&sm->o_done[j][i], 1);
      }
      mbar_init(&sm->plan_full[j], 1);
      mbar_init(&sm->plan_empty[j], 2 * kQ + 128 + 2);
    }
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 12) tmem_alloc(&sm->tmem, kTmemCols);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int parts = SHARED ? int(cluster_size()) : 1, part = SHARED ? int(cluster_rank()) : 0;
  tc_fence_before();
  if (SHARED) cluster_sync();  // barriers that others arrive at
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, sm->tmem, 0);
  const int P = gridDim.x / parts, ci = blockIdx.x / parts;
  // Every wait is bounded; a role that gives up leaves its loop, the others follow when their own waits run out.
  bool ok = true;
  auto ring_wait = [&](uint64_t* bars, int n) { return mbar_wait(&bars[n & (kRing - 1)], uint32_t(n / kRing) & 1u); };
  auto pair_wait = [&](uint64_t* bars, int c) { return mbar_wait(&bars[c & 1], uint32_t(c >> 1) & 1u); };

  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 13) {
      // -------------------------------------------------------------- plans
      for (int u = ci, k = 0; u < units; u += P, ++k) {
        if (k >= 2) ok = __all_sync(kFull, pair_wait(sm->plan_empty, k - 2));
        if (!ok) break;
        plan_unit(a, &sm->plan[k & 1], u, rows_per, part == 0, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->plan_full[k & 1]);
      }
    } else if (warp != 15) {
      // -------------------------------------------------------------- products: of warpgroup j's scores
      const int j = warp == 14;
      const bool leader = elect_one();
      const uint32_t q_addr = smem_u32(sm->q), st_addr = smem_u32(sm->st);
      int n0 = 0, c0 = 0, seg = 0;  // tiles and jobs before this pass
      for (int u = ci, k = 0; u < units && ok; u += P, ++k) {
        ok = pair_wait(sm->plan_full, k);
        const Plan& plan = sm->plan[k & 1];
        for (int ps = 0; ok && ps < plan.passes; ++ps, ++seg) {
          const Walk g = walk_of(a, plan, ps, part, parts);
          ok = mbar_wait(&sm->q_full, uint32_t(seg) & 1u);
          const int jobs = jobs_of(g, j);
          const uint64_t qd = tile_desc(q_addr + (g.both ? j : 0) * uint32_t(sizeof(sm->q[0])));
          // P . V runs one job behind the scores
          for (int i = 0; i <= jobs && ok; ++i) {
            if (i < jobs) {
              const int n = n0 + (g.both ? i : 2 * i + j), c = c0 + i;
              ok = ring_wait(sm->full, n);
              if (c >= 2) ok = ok && pair_wait(sm->o_done[j], c - 2);  // S's buffer: its weights have been read
              if (!ok) break;
              tc_fence_after();
              const uint64_t kd = tile_desc(st_addr + uint32_t(n & (kRing - 1)) * uint32_t(sizeof(TcStage)));
              const uint32_t d = tmem + 256 + 128 * j + 64 * (c & 1);
              if (leader) {
#pragma unroll
                for (int e = 0; e < kHeadDim / 16; ++e)
                  tc_mma_ss(d, qd + (e >> 2) * (sizeof(sm->q[0][0]) >> 4) + 2 * (e & 3),
                            kd + (e >> 2) * (sizeof(sm->st[0].k[0]) >> 4) + 2 * (e & 3), f16_idesc(kQ, kTok), e > 0);
                if constexpr (TWO) {
#pragma unroll
                  for (int e = 0; e < kHeadDim / 16; ++e)
                    tc_mma_ss(d, qd + (sizeof(sm->q[0]) >> 4) + (e >> 2) * (sizeof(sm->q[0][0]) >> 4) + 2 * (e & 3),
                              kd + (e >> 2) * (sizeof(sm->st[0].k[0]) >> 4) + 2 * (e & 3), f16_idesc(kQ, kTok), true);
                }
                tc_commit(&sm->s_full[j][c & 1]);
              }
              __syncwarp();
            }
            if (i > 0) {
              const int n = n0 + (g.both ? i - 1 : 2 * (i - 1) + j), s = n & (kRing - 1), c = c0 + i - 1;
              const uint64_t vd =
                  tile_desc(st_addr + uint32_t(s) * uint32_t(sizeof(TcStage)) + uint32_t(sizeof(sm->st[0].k)));
              const uint32_t d = tmem + 128 * j, w = tmem + 256 + 128 * j + 64 * (c & 1);
              ok = pair_wait(sm->p_full[j], c);
              if (!ok) break;
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int e = 0; e < kTok / 16; ++e)
                  tc_mma_ts(d, w + 8 * e, vd + 2 * e, f16_idesc(kQ, kHeadDim), i > 1 || e > 0);
                tc_commit(&sm->o_done[j][c & 1]);
                tc_commit(&sm->empty[s]);
                if (!g.both) tc_commit(&sm->empty[s]);  // for the other warpgroup, which this tile passes by
              }
              __syncwarp();
            }
          }
          n0 += g.nt;
          c0 += jobs;
        }
        if (lane == 0) mbar_arrive(&sm->plan_empty[k & 1]);
      }
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- conversion
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    const int w = warp - 8;
    const uint32_t km = magic_f16x2(a.B);
    const uint32_t c64 = 0x64646464u | (uint32_t(a.B) >> 16);  // a.B <= 4096: the constant itself
    int n = 0, seg = 0;
    for (int u = ci, k = 0; u < units && ok; u += P, ++k) {
      ok = __all_sync(kFull, pair_wait(sm->plan_full, k));
      if (!ok) break;
      const Plan& plan = sm->plan[k & 1];
      for (int ps = 0; ok && ps < plan.passes; ++ps, ++seg) {
        const Walk g = walk_of(a, plan, ps, part, parts);
        if (SHARED && seg > 0) {  // the ring holds the state that the cluster reads
          ok = __all_sync(kFull, cluster_wait(&sm->release, uint32_t(seg - 1) & 1u));
          if (!ok) break;
        }
        const int* table = a.table + size_t(g.seq) * a.mbps;
        int ids = -1, ids_next = -1;  // this warp's table entries of 32 tiles, and of the next 32
        uint32_t show = 0xFFFFu, show_next = 0xFFFFu;  // which of their tokens are seen, where rows are apart
        auto load_ids = [&](int i) {
          const int blk = g.tile(i + lane) * kStep + w;
          int id = -1;
          bool seen = i + lane < g.nt && blk * kBlock < g.most && (blk * kBlock < a.sinks || (blk + 1) * kBlock > g.from);
          if (g.apart && seen) {
            show_next = seen_tokens(plan, g.seq, blk, a.sinks, a.span);
            seen = show_next != 0;
          }
          if (seen) {
            id = __ldcg(table + blk);
            if (id < 0 || id >= a.c.num_blocks) {
              flag(a.err, KVQ_DEVERR_BLOCK_ID);
              id = 0;
            }
          }
          return id;
        };
        ids_next = load_ids(0);
        // this warp's block of the tile: codes, and the record entries of token `lane` (lanes 0..15)
        Raw<KB> rk;
        Raw<VB> rv;
        float ks = 0.f, vs = 0.f, ko = 0.f, vo = 0.f;
        auto block_of = [&](int i) {  // called once per tile, in order
          if ((i & 31) == 0) {
            ids = ids_next;
            show = show_next;
            ids_next = load_ids(i + 32);
          }
          return i < g.nt ? __shfl_sync(kFull, ids, i & 31) : -1;
        };
        auto fetch_keys = [&](int phys) {
          ks = vs = ko = vo = 0.f;
          rk.clear();
          if (phys < 0) return;
          const size_t hb = size_t(g.h) * a.c.num_blocks + phys;
          rk.load(a.c.k_codes + hb * F::kKBB, lane);
          const float* rec = a.c.meta + hb * F::kMF + (F::kGroup ? 0 : (lane & 15));
          ks = a.c.k_chan ? 1.f : __ldcg(rec + F::kKS);
          vs = __ldcg(rec + F::kVS);
          if constexpr (ASYM) {
            ko = __ldcg(rec + F::kKO);
            vo = __ldcg(rec + F::kVO);
          }
        };
        auto fetch_values = [&](int phys) {
          rv.clear();
          if (phys >= 0) rv.load(a.c.v_codes + (size_t(g.h) * a.c.num_blocks + phys) * F::kVBB, lane);
        };
        {
          const int phys = block_of(0);
          fetch_keys(phys);
          fetch_values(phys);
        }
#pragma unroll 1
        for (int i = 0; i < g.nt; ++i, ++n) {
          const int s = n & (kRing - 1);
          ok = __all_sync(kFull, n < kRing || ring_wait(sm->empty, n - kRing));
          if (!ok) break;
          put_keys<KB>(rk, sm->st[s].k[0], sm->st[s].k[1], w, lane, km, c64);
          const int pos = (g.tile(i) * kStep + w) * kBlock + lane;
          bool data = pos < g.most && (pos < a.sinks || pos >= g.from);
          if (g.apart) {
            const uint32_t tokens = __shfl_sync(kFull, show, i & 31);
            data = data && (tokens >> (lane & 15) & 1u);
          }
          if (!data) vs = 0.f;
          if (lane < kBlock) {
            const int col = tile_col(w, lane);
            sm->sk[s][col] = ks * kUnitScale;
            sm->sv[s][col] = vs;
            if constexpr (ASYM) {
              sm->mk[s][col] = fmaf(kKC, ks, ko) * kUnitScale;
              sm->mv[s][col] = data ? fmaf(kVC, vs, vo) : 0.f;
            }
          }
          // value scales are positive: they order as their bits
          const uint32_t vm = __reduce_max_sync(kFull, lane < kBlock ? __float_as_uint(vs) : 0u);
          if (lane == 0) sm->svmax[s][w] = __uint_as_float(vm);
          const int phys = block_of(i + 1);
          fetch_keys(phys);
          put_values<VB>(rv, sm->st[s].v, w, lane, km, c64);
          fetch_values(phys);
          fence_async_smem();
          mbar_arrive(&sm->full[s]);
        }
      }
      mbar_arrive(&sm->plan_empty[k & 1]);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");  // 256 x 176 + 128 x (96 + 64): the launch's 512 x 128
    const int j = warp >> 2, v = tid & (kQ - 1);  // warpgroup, its vector
    const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t o_cols = lanes + 128 * j, s_cols = lanes + 256 + 128 * j;
    int n0 = 0, c = 0, seg = 0;  // tiles before this pass; this warpgroup's jobs so far
    uint32_t meets = 0;
    auto meet = [&]() {  // both warpgroups
      mbar_arrive(&sm->meet);
      return __all_sync(kFull, mbar_wait(&sm->meet, meets++ & 1u)) != 0;
    };
    for (int u = ci, k = 0; u < units && ok; u += P, ++k) {
      ok = __all_sync(kFull, pair_wait(sm->plan_full, k));
      if (!ok) break;
      const Plan& plan = sm->plan[k & 1];
      for (int ps = 0; ok && ps < plan.passes; ++ps, ++seg) {
        const Walk g = walk_of(a, plan, ps, part, parts);
        if (seg > 0 && !(ok = meet())) break;  // both are done with the previous pass's queries
        if (SHARED && seg > 0) {
          ok = __all_sync(kFull, cluster_wait(&sm->release, uint32_t(seg - 1) & 1u));
          if (!ok) break;
        }
        const int G = a.G;
        {
          // this warp's 32 vectors (16 of the shared 128), 4 a step
          const int per = g.both ? 32 : 16, v0 = (g.both ? warp : 2 * (warp & 3) + j) * per, sub = lane & 7;
          const uint16_t* src = a.q + (size_t(plan.r0) * a.Hq + g.h * G) * kHeadDim + 16 * sub;
          float f[16];
          if (a.c.factor) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(f + e) =
                  __ldcg(reinterpret_cast<const float4*>(a.c.factor + g.h * kHeadDim + 16 * sub + e));
          }
          uint8_t* half = sm->q[g.both ? j : 0][sub & 1];
          int r = (v0 + (lane >> 3)) / G, hj = (v0 + (lane >> 3)) % G;
          uint4 raw[8][2];  // all loads before the first conversion: one latency
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
            if (4 * i < per && r < plan.nrows) {
              const uint4* p = reinterpret_cast<const uint4*>(src + (size_t(r) * a.Hq + hj) * kHeadDim);
              raw[i][0] = __ldcg(p);
              raw[i][1] = __ldcg(p + 1);
            }
            hj += 4;
            while (hj >= G) {
              hj -= G;
              ++r;
            }
          }
          if (lane < per) {
            const int row = (v0 + lane) / G;
            sm->qlen[v0 + lane] = row < plan.nrows && plan.seq[row] == g.seq ? plan.len[row] : 0;
          }
          // queries as they are, of ordinary size (most passes): scaled by 2^kFixedExp and rounded, eight vectors a step
          bool plain = !TWO && a.c.q_bits == 16 && !a.c.factor;
          if (plain) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t w = 0u;
#pragma unroll
              for (int x = 0; x < 2; ++x)
                w = __vmaxu2(__vmaxu2(w, __vmaxu2(raw[i][x].x & kAbs2, raw[i][x].y & kAbs2)),
                             __vmaxu2(raw[i][x].z & kAbs2, raw[i][x].w & kAbs2));
              w = max(w & 0xFFFFu, w >> 16);  // a lane's 16 values; a lane of zeros (its vector's other lanes decide) is plain
              plain = plain && (w == 0u || w - kLeastBits <= kMostBits - kLeastBits);
            }
            plain = __all_sync(kFull, plain);
          }
          if (plain) {
#pragma unroll 1
            for (int b = 0; b < per; b += 8) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int at = v0 + b + 4 * e + (lane >> 3);
                const float sum = put_plain<ASYM>(raw[e], half, at & (kQ - 1), sub);
                if (sub == 0) {
                  sm->qs[at] = 1.f;
                  sm->qz[at] = sum;
                }
              }
#pragma unroll
              for (int e = 0; e < 6; ++e) {
                raw[e][0] = raw[e + 2][0];
                raw[e][1] = raw[e + 2][1];
              }
            }
          }
#pragma unroll 1
          for (int b = plain ? per : 0; b < per; b += 4) {
            const uint4 cur[2] = {raw[0][0], raw[0][1]};
#pragma unroll
            for (int e = 0; e < 7; ++e) {  // rotate: the loop stays short and every index is known
              raw[e][0] = raw[e + 1][0];
              raw[e][1] = raw[e + 1][1];
            }
            const int at = v0 + b + (lane >> 3);
            float qs, sum;
            put_query<ASYM, TWO, true>(a, cur, f, half, int(sizeof(sm->q[0])), at & (kQ - 1), sub, qs, sum);
            if (sub == 0) {
              sm->qs[at] = qs;
              sm->qz[at] = sum;
            }
          }
        }
        fence_async_smem();
        mbar_arrive(&sm->q_full);
        ok = __all_sync(kFull, mbar_wait(&sm->q_full, uint32_t(seg) & 1u));
        if (!ok) break;
        // Of its warp's 32 rows a thread holds four, lane / 4 + 8 b, and of their scores two columns of every eight,
        // 8 n + 2 (lane % 4) and the next (the fragments of 16-lane tensor-memory accesses): a scale that is read serves four rows.
        const int base_v = g.both ? warp * 32 : (warp & 3) * 32, t = lane & 3;
        float l[4][2], z[4], qz[4];  // l: two partial sums of the weights
        float nb[4], thr[4];  // sigma - m; the exponent from which on the maximum has to move
        float svlim = ldexpf(1.f, kWeightExp - int(kMaxSlack) - kSigma0);  // the largest value scale that all four rows allow
        uint32_t nan_rows = 0;  // rows whose outputs are no numbers
        bool scaled = false;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int at = base_v + (lane >> 2) + 8 * b;
          scaled |= sm->qs[at] != 1.f;
          qz[b] = ASYM ? sm->qz[at] * sm->qs[at] : 0.f;
          thr[b] = kNegInf;
          l[b][0] = l[b][1] = z[b] = nb[b] = 0.f;
          sm->rm[warp * 32 + (lane >> 2) + 8 * b] = kNegInf;
          sm->rl[warp * 32 + (lane >> 2) + 8 * b] = float(kSigma0);
        }
        scaled = __any_sync(kFull, scaled);
        const int len = sm->qlen[base_v + lane];  // of the row that this thread writes
        // the warp's shortest row and latest window decide whether a tile needs the mask at all (vectors that are not of
        // this pass do not count)
        const int minlen = __reduce_min_sync(kFull, len > 0 ? len : 0x7fffffff);
        const int maxlo = __reduce_max_sync(kFull, len > 0 ? len - a.span : -0x7fffffff);
        const int jobs = jobs_of(g, j);
#pragma unroll 1
        for (int i = 0; i < jobs; ++i, ++c) {
          const int tile = g.both ? i : 2 * i + j, sc = (n0 + tile) & (kRing - 1);
          // the tile's scales are asked for before its scores: shared memory takes some 300 cycles to answer beside the
          // products' reads
          ok = __all_sync(kFull, ring_wait(sm->full, n0 + tile));
          if (!ok) break;
          const float4 sm4 = *reinterpret_cast<const float4*>(sm->svmax[sc]);
          float2 ks[8], ko[8], vs[8], vo[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            ks[n] = *reinterpret_cast<const float2*>(&sm->sk[sc][8 * n + 2 * t]);
            if constexpr (ASYM) ko[n] = *reinterpret_cast<const float2*>(&sm->mk[sc][8 * n + 2 * t]);
            else vs[n] = *reinterpret_cast<const float2*>(&sm->sv[sc][8 * n + 2 * t]);
          }
          ok = __all_sync(kFull, pair_wait(sm->s_full[j], c));
          if (!ok) break;
          tc_fence_after();
          const uint32_t st = s_cols + 64 * (c & 1);
          uint32_t r[2][32];  // rows 16 h ..: score (n, e, x) of row 16 h + lane / 4 + 8 e, column 8 n + 2 t + x at 4 n + 2 e + x
          tmem_ld16(st, r[0]);
          tmem_ld16(st + (16u << 16), r[1]);
          tc_wait_ld();
          const int tok0 = g.tile(tile) * kTok;
          if (scaled) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const float qs = sm->qs[base_v + (lane >> 2) + 8 * b];
#pragma unroll
              for (int n = 0; n < 8; ++n) mul2(r[b >> 1][4 * n + 2 * (b & 1)], r[b >> 1][4 * n + 2 * (b & 1) + 1], qs, qs);
            }
          }
#pragma unroll
          for (int n = 0; n < 8; ++n) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              uint32_t &x = r[b >> 1][4 * n + 2 * (b & 1)], &y = r[b >> 1][4 * n + 2 * (b & 1) + 1];
              if constexpr (ASYM) {
                uint32_t bx = __float_as_uint(ko[n].x), by = __float_as_uint(ko[n].y);
                fma2(bx, by, qz[b], qz[b], nb[b], nb[b]);
                fma2(x, y, ks[n].x, ks[n].y, __uint_as_float(bx), __uint_as_float(by));
              } else {
                fma2(x, y, ks[n].x, ks[n].y, nb[b], nb[b]);
              }
            }
          }
          auto value_scales = [&]() {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              vs[n] = *reinterpret_cast<const float2*>(&sm->sv[sc][8 * n + 2 * t]);
              if constexpr (ASYM) vo[n] = *reinterpret_cast<const float2*>(&sm->mv[sc][8 * n + 2 * t]);
            }
          };
          if constexpr (ASYM) value_scales();
          // a row of the warp that ends inside this tile or before it, or hides tokens of it.  Column (n, x) of this
          // thread is token 16 (n % 4) + 4 (n / 4) + t + 8 x of the tile
          const bool masked = tok0 + kTok > minlen || (tok0 < maxlo && tok0 + kTok > a.sinks);
          if (masked) {
            const int first = a.sinks - tok0 - t;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int own = sm->qlen[base_v + (lane >> 2) + 8 * b], left = own - tok0 - t, hidden = max(own - a.span - a.sinks, 0);
#pragma unroll
              for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int off = 16 * (n & 3) + 4 * (n >> 2) + 8 * x;
                  if (off >= left || unsigned(off - first) < unsigned(hidden))
                    r[b >> 1][4 * n + 2 * (b & 1) + x] = __float_as_uint(kNegInf);
                }
            }
          }
          float mx[4];
          bool over = false;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            float x2[2] = {kNegInf, kNegInf};
#pragma unroll
            for (int n = 0; n < 8; ++n)
              x2[n & 1] = max3(x2[n & 1], __uint_as_float(r[b >> 1][4 * n + 2 * (b & 1)]),
                               __uint_as_float(r[b >> 1][4 * n + 2 * (b & 1) + 1]));
            mx[b] = fmaxf(x2[0], x2[1]);
            over |= mx[b] > thr[b];
          }
          const float svm = max_nan(max_nan(sm4.x, sm4.y), max_nan(sm4.z, sm4.w));  // the same in every thread
          if (__any_sync(kFull, over || !(svm <= svlim))) {
            float f[4] = {1.f, 1.f, 1.f, 1.f}, m[4], sg[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              m[b] = sm->rm[warp * 32 + (lane >> 2) + 8 * b];
              sg[b] = sm->rl[warp * 32 + (lane >> 2) + 8 * b];
            }
            __syncwarp();
            if (__any_sync(kFull, over)) {
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                mx[b] = fmaxf(mx[b], __shfl_xor_sync(kFull, mx[b], 1));
                mx[b] = fmaxf(mx[b], __shfl_xor_sync(kFull, mx[b], 2));
                const float mn = fmaxf(m[b], mx[b] - nb[b]);  // every row's: one at a time, they would come back often (195 us)
                f[b] = mn == kNegInf ? 1.f : ex2(m[b] - mn);
                m[b] = mn;
              }
            }
            if (__any_sync(kFull, !(svm <= svlim))) {
              if (!(svm <= kFloatMax)) {
                // A value scale that is not finite: -1 stands for it, as in rows that do not see its token 0 x inf would be
                // no number.  Every warp that goes on to use the scales writes the same.
                for (int e = lane; e < kTok; e += 32)
                  if (!(fabsf(sm->sv[sc][e]) <= kFloatMax)) {
                    sm->sv[sc][e] = -1.f;
                    if constexpr (ASYM) sm->mv[sc][e] = 0.f;
                  }
                __syncwarp();
                value_scales();
              }
              // by the scales that each row sees: of this thread's columns, then of the row's four threads
              float sv[4] = {0.f, 0.f, 0.f, 0.f}, least[4] = {0.f, 0.f, 0.f, 0.f};
              int own[4];
#pragma unroll
              for (int b = 0; b < 4; ++b) own[b] = sm->qlen[base_v + (lane >> 2) + 8 * b];
              const int first = a.sinks - tok0 - t;
#pragma unroll
              for (int b = 0; b < 4; ++b) sv[b] = own[b] > 0 && !masked && svm <= kFloatMax ? svm : 0.f;
#pragma unroll 1
              for (int n = masked || !(svm <= kFloatMax) ? 0 : 8; n < 8; ++n) {
                const float2 s2 = *reinterpret_cast<const float2*>(&sm->sv[sc][8 * n + 2 * t]);
                const int off = 16 * (n & 3) + 4 * (n >> 2);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  const int left = own[b] - tok0 - t, hidden = max(own[b] - a.span - a.sinks, 0);
                  const float s0 = off >= left || unsigned(off - first) < unsigned(hidden) ? 0.f : s2.x;
                  const float s1 = off + 8 >= left || unsigned(off + 8 - first) < unsigned(hidden) ? 0.f : s2.y;
                  sv[b] = fmaxf(sv[b], fmaxf(s0, s1));
                  least[b] = fminf(least[b], fminf(s0, s1));
                }
              }
              svlim = kFloatMax;
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                sv[b] = fmaxf(sv[b], __shfl_xor_sync(kFull, sv[b], 1));
                sv[b] = fmaxf(sv[b], __shfl_xor_sync(kFull, sv[b], 2));
                least[b] = fminf(least[b], __shfl_xor_sync(kFull, least[b], 1));
                least[b] = fminf(least[b], __shfl_xor_sync(kFull, least[b], 2));
                if (least[b] < 0.f) nan_rows |= 1u << b;
                // sigma down to what the row's largest scale asks for (below 2^e, normal wherever it asks)
                const int e = int(__float_as_uint(sv[b]) >> 23) - 126, s0 = int(sg[b]);
                const int sn = min(s0, kWeightExp - int(kMaxSlack) - e);
                f[b] *= pow2(sn - s0);
                sg[b] = float(sn);
                // a row that has ended, is not of this pass, or is no number has no more say
                if (own[b] > tok0 && !(nan_rows >> b & 1u)) svlim = fminf(svlim, pow2(kWeightExp - int(kMaxSlack) - sn));
              }
            }
            float fo = 1.f;  // of the row whose O this thread holds: lane
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              sm->rm[warp * 32 + (lane >> 2) + 8 * b] = m[b];  // all four threads of the row
              sm->rl[warp * 32 + (lane >> 2) + 8 * b] = sg[b];
              const float was = nb[b];
              nb[b] = m[b] == kNegInf ? 0.f : sg[b] - m[b];
              thr[b] = m[b] == kNegInf ? kNegInf : kMaxSlack + sg[b];
              const uint32_t by = __float_as_uint(nb[b] - was);
#pragma unroll
              for (int n = 0; n < 8; ++n) add2(r[b >> 1][4 * n + 2 * (b & 1)], r[b >> 1][4 * n + 2 * (b & 1) + 1], by, by);
              l[b][0] *= f[b];
              l[b][1] *= f[b];
              z[b] *= f[b];
              const float fb = __shfl_sync(kFull, f[b], 4 * (lane & 7));
              fo = (lane >> 3) == b ? fb : fo;
            }
            if (i > 0) {  // O too, once the products so far are complete
              ok = __all_sync(kFull, pair_wait(sm->o_done[j], c - 1));
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int e = 0; e < kHeadDim; e += 32) {
                uint32_t o[32];
                tmem_ld32(o_cols + e, o);
                tc_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * fo);
                tmem_st32(o_cols + e, o);
              }
              tc_wait_st();
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 16 rows, stored while the next are at work
            uint32_t p[16];
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int b = 2 * h + e;
                uint32_t x = __float_as_uint(ex2(__uint_as_float(r[h][4 * n + 2 * e])));
                uint32_t y = __float_as_uint(ex2(__uint_as_float(r[h][4 * n + 2 * e + 1])));
                uint32_t &l0 = reinterpret_cast<uint32_t&>(l[b][0]), &l1 = reinterpret_cast<uint32_t&>(l[b][1]);
                add2(l0, l1, x, y);
                if constexpr (ASYM) z[b] = fmaf(__uint_as_float(x), vo[n].x, fmaf(__uint_as_float(y), vo[n].y, z[b]));
                mul2(x, y, vs[n].x, vs[n].y);
                p[2 * n + e] = pack_half2(__uint_as_float(x), __uint_as_float(y));
              }
            tmem_st16x128(st + (uint32_t(16 * h) << 16), p);  // over S, which has been read
          }
          tc_wait_st();
          tc_fence_before();
          mbar_arrive(&sm->p_full[j][c & 1]);
        }
        if (!ok) break;
        // ---- the pass's outputs
        if (jobs > 0) {
          ok = __all_sync(kFull, pair_wait(sm->o_done[j], c - 1));
          if (!ok) break;
          tc_fence_after();
        }
        // the state of row `lane`, from its four threads: exponent base, sum, what is added to each output
        __syncwarp();
        float row_m = sm->rm[warp * 32 + lane], row_l = 0.f, add = 0.f;
        if (row_m != kNegInf) row_m -= sm->rl[warp * 32 + lane];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          float lb = l[b][0] + l[b][1], zb = z[b];
          lb += __shfl_xor_sync(kFull, lb, 1);
          lb += __shfl_xor_sync(kFull, lb, 2);
          if constexpr (ASYM) {
            zb += __shfl_xor_sync(kFull, zb, 1);
            zb += __shfl_xor_sync(kFull, zb, 2);
          }
          if (nan_rows >> b & 1u) zb = __int_as_float(0x7fffffff);
          lb = __shfl_sync(kFull, lb, 4 * (lane & 7));
          zb = __shfl_sync(kFull, zb, 4 * (lane & 7));
          if ((lane >> 3) == b) {
            row_l = lb;
            add = zb;
          }
        }
        // row i of the warp: its place, or -1 (its own thread's length)
        const size_t out0 = size_t(plan.r0) * a.Hq + g.h * G;
        auto place = [&](int vec) { return (out0 + size_t(vec / G) * a.Hq + vec % G) * kHeadDim; };
        const uint32_t used = __ballot_sync(kFull, len > 0);
        float4* buf;
        float4* const state = reinterpret_cast<float4*>(sm->st);  // [vector][32 chunks of 4], chunks by the vector's lane
        if (SHARED && g.both) {
          ok = meet();  // the ring is drained once both have seen their last products
          if (!ok) break;
          sm->rm[tid] = row_m;
          sm->rl[tid] = row_l;
          if (jobs > 0) {
#pragma unroll 1
            for (int e = 0; e < kHeadDim; e += 32) {
              uint32_t o[32];
              tmem_ld32(o_cols + e, o);
              tc_wait_ld();
#pragma unroll
              for (int b = 0; b < 8; ++b)
                state[tid * 32 + ((e / 4 + b) ^ lane)] =
                    make_float4(__uint_as_float(o[4 * b]) + add, __uint_as_float(o[4 * b + 1]) + add,
                                __uint_as_float(o[4 * b + 2]) + add, __uint_as_float(o[4 * b + 3]) + add);
            }
          }
        } else if (g.both) {
          // by way of 4 KB of this warp's in its own Q, which no product reads any more
          buf = reinterpret_cast<float4*>(sm->q[j][0]) + (warp & 3) * 256;
          const float inv = 1.f / row_l;
          if (len > 0 && a.lse) a.lse[place(tid) / kHeadDim] = (row_m + log2f(row_l)) * kLn2;
          size_t to[8];  // of the rows that this lane writes
#pragma unroll
          for (int b = 0; b < 8; ++b) to[b] = place(warp * 32 + 4 * b + (lane >> 3)) + 4 * (lane & 7);
#pragma unroll 1
          for (int e = 0; e < kHeadDim; e += 32) {
            uint32_t o[32];
            tmem_ld32(o_cols + e, o);
            tc_wait_ld();
#pragma unroll
            for (int b = 0; b < 8; ++b)
              buf[lane * 8 + (b ^ (lane & 7))] =
                  make_float4((__uint_as_float(o[4 * b]) + add) * inv, (__uint_as_float(o[4 * b + 1]) + add) * inv,
                              (__uint_as_float(o[4 * b + 2]) + add) * inv, (__uint_as_float(o[4 * b + 3]) + add) * inv);
            __syncwarp();
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              const int row = 4 * b + (lane >> 3);
              if (used >> row & 1u)
                put_out(a, to[b] + e, buf[row * 8 + ((lane & 7) ^ (row & 7))]);
            }
            __syncwarp();
          }
        } else {
          // both hold the same vectors: the second one's state goes through Q once every product of the pass is done
          ok = meet();
          if (!ok) break;
          buf = reinterpret_cast<float4*>(sm->q[0][0]) + v * 32;  // this vector's 128 values, chunks by its lane
          if (j == 1) {
            sm->qs[v] = row_m;
            sm->qz[v] = row_l;
            if (jobs > 0) {
#pragma unroll 1
              for (int e = 0; e < kHeadDim; e += 32) {
                uint32_t o[32];
                tmem_ld32(o_cols + e, o);
                tc_wait_ld();
#pragma unroll
                for (int b = 0; b < 8; ++b)
                  buf[(e / 4 + b) ^ lane] =
                      make_float4(__uint_as_float(o[4 * b]) + add, __uint_as_float(o[4 * b + 1]) + add,
                                  __uint_as_float(o[4 * b + 2]) + add, __uint_as_float(o[4 * b + 3]) + add);
              }
            }
          }
          ok = meet();
          if (!ok) break;
          if (j == 0) {
            const float m0 = row_m, m1 = sm->qs[v];
            const float M = fmaxf(m0, m1);
            const float w0 = m0 == kNegInf ? 0.f : exp2f(m0 - M), w1 = m1 == kNegInf ? 0.f : exp2f(m1 - M);
            const float L = w0 * row_l + w1 * sm->qz[v], inv = 1.f / L;
            // a warpgroup without a tile has left no values; one that is no number stays none
            const bool other = jobs_of(g, 1) > 0, here = jobs > 0;
            const float scale = SHARED ? 1.f : inv;
            if constexpr (SHARED) {
              sm->rm[v] = M;
              sm->rl[v] = L;
              buf = state + v * 32;
            } else if (len > 0 && a.lse) {
              a.lse[place(v) / kHeadDim] = (M + log2f(L)) * kLn2;
            }
            const float4* from = reinterpret_cast<const float4*>(sm->q[0][0]) + v * 32;
#pragma unroll 1
            for (int e = 0; e < kHeadDim; e += 32) {
              uint32_t o[32];
              tmem_ld32(o_cols + e, o);
              tc_wait_ld();
#pragma unroll
              for (int b = 0; b < 8; ++b) {
                const float4 y = other ? from[(e / 4 + b) ^ lane] : make_float4(0.f, 0.f, 0.f, 0.f);
                if (!here) o[4 * b] = o[4 * b + 1] = o[4 * b + 2] = o[4 * b + 3] = 0u;
                buf[(e / 4 + b) ^ lane] = make_float4((w0 * (__uint_as_float(o[4 * b]) + add) + w1 * y.x) * scale,
                                                      (w0 * (__uint_as_float(o[4 * b + 1]) + add) + w1 * y.y) * scale,
                                                      (w0 * (__uint_as_float(o[4 * b + 2]) + add) + w1 * y.z) * scale,
                                                      (w0 * (__uint_as_float(o[4 * b + 3]) + add) + w1 * y.w) * scale);
              }
            }
            __syncwarp();
            const float4* rows = reinterpret_cast<const float4*>(sm->q[0][0]) + warp * 32 * 32;
            for (int row = 0; !SHARED && row < 32; ++row)
              if (used >> row & 1u) put_out(a, place(warp * 32 + row) + 4 * lane, rows[row * 32 + (lane ^ row)]);
          }
        }
        if constexpr (SHARED) {
          // ---- the cluster's shares of each vector, this CTA's part of the vectors: four of them a step of a warp, whose
          // states are all on their way at once
          for (int r = 0; r < parts; ++r) remote_arrive(&sm->gather, r);
          ok = __all_sync(kFull, cluster_wait(&sm->gather, uint32_t(seg) & 1u));
          if (!ok) break;
          const int log_p = 31 - __clz(parts), mine = lane >> log_p, share = lane & (parts - 1);
          for (int base = 4 * warp; base * parts < g.nv; base += 32) {
            // vector part + parts * (base + i); lanes i * parts + r hold its m and l in share r
            const int own = part + parts * (base + mine);
            const bool in = mine < 4 && own < g.nv;
            const float m_of = in ? remote_float(&sm->rm[own], share) : kNegInf;
            float M = m_of, L = in ? remote_float(&sm->rl[own], share) : 0.f;
            for (int o = parts >> 1; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
            const float weight = m_of == kNegInf ? 0.f : exp2f(m_of - M);
            L *= weight;
            for (int o = parts >> 1; o > 0; o >>= 1) L += __shfl_xor_sync(kFull, L, o);
            float4 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int r = 0; r < parts; ++r) {
              float4 x[4];
              float w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int vec = part + parts * (base + i), at = (i << log_p) + r;
                w[i] = __shfl_sync(kFull, weight, at);
                // a share that saw nothing, or had no tile, has left no values
                const bool left = vec < g.nv && __shfl_sync(kFull, m_of, at) != kNegInf;
                x[i] = left ? remote_float4(state + vec * 32 + (lane ^ (vec & 31)), r) : make_float4(0.f, 0.f, 0.f, 0.f);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[i].x = fmaf(w[i], x[i].x, o[i].x);
                o[i].y = fmaf(w[i], x[i].y, o[i].y);
                o[i].z = fmaf(w[i], x[i].z, o[i].z);
                o[i].w = fmaf(w[i], x[i].w, o[i].w);
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int vec = part + parts * (base + i);
              const float Lv = __shfl_sync(kFull, L, i << log_p), Mv = __shfl_sync(kFull, M, i << log_p), inv = 1.f / Lv;
              if (vec >= g.nv || sm->qlen[vec] == 0) continue;
              const size_t at = place(vec);
              put_out(a, at + 4 * lane, make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv));
              if (lane == 0 && a.lse) a.lse[at / kHeadDim] = (Mv + log2f(Lv)) * kLn2;
            }
          }
          for (int r = 0; r < parts; ++r) remote_arrive(&sm->release, r);
        }
        tc_fence_before();
        n0 += g.nt;
      }
      mbar_arrive(&sm->plan_empty[k & 1]);
    }
  }
  if (!ok) flag(a.err, KVQ_DEVERR_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  if (SHARED) cluster_sync();  // the others may still read this CTA's shared memory
  else __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_free(tmem, kTmemCols);
}

// The kernel of one format, as a cluster of 2^c CTAs a unit takes it (c 0: one CTA a unit, units in turn).
template <int KB, int VB, bool ASYM, bool TWO, bool SHARED>
struct UnitKernel {
  static constexpr int kSmem = int(sizeof(UnitSmem)) + 1024;
  static_assert(kSmem <= 232448, "shared memory of an SM");
  static cudaError_t prepare() {
    return cudaFuncSetAttribute(sinks_tc_kernel<KB, VB, ASYM, TWO, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmem);
  }
  static cudaLaunchConfig_t config(int ctas, int c, cudaLaunchAttribute (&attr)[2], cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(ctas));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1u << c;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c > 0 ? 2 : 1;
    return cfg;
  }
  static cudaError_t clusters(int ctas, int c, int* n) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config(ctas, c, attr, nullptr);
    return cudaOccupancyMaxActiveClusters(n, sinks_tc_kernel<KB, VB, ASYM, TWO, SHARED>, &cfg);
  }
  static cudaError_t launch(const DecodeArgs& a, int units, int rows, int ctas, int c, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config(ctas, c, attr, s);
    return cudaLaunchKernelEx(&cfg, sinks_tc_kernel<KB, VB, ASYM, TWO, SHARED>, a, units, rows);
  }
};

template <bool TWO, bool SHARED, class F>
cudaError_t by_bits(const CacheView& v, F f) {
  const int kb = v.k_bits, vb = v.v_bits;
  const bool as = v.asym != 0;
  if (kb == 8 && vb == 8) return as ? f(UnitKernel<8, 8, true, TWO, SHARED>{}) : f(UnitKernel<8, 8, false, TWO, SHARED>{});
  if (kb == 4 && vb == 4) return as ? f(UnitKernel<4, 4, true, TWO, SHARED>{}) : f(UnitKernel<4, 4, false, TWO, SHARED>{});
  if (kb == 4 && vb == 8) return as ? f(UnitKernel<4, 8, true, TWO, SHARED>{}) : f(UnitKernel<4, 8, false, TWO, SHARED>{});
  if (kb == 8 && vb == 4) return as ? f(UnitKernel<8, 4, true, TWO, SHARED>{}) : f(UnitKernel<8, 4, false, TWO, SHARED>{});
  return as ? f(UnitKernel<2, 2, true, TWO, SHARED>{}) : f(UnitKernel<2, 2, false, TWO, SHARED>{});
}

template <bool SHARED, class F>
cudaError_t by_format(const CacheView& v, F f) {
  return v.q_bits == 32 ? by_bits<true, SHARED>(v, f) : by_bits<false, SHARED>(v, f);
}

}  // namespace
}  // namespace kvq
