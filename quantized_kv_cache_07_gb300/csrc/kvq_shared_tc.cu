// The shared prefix of kvq_decode_shared on tcgen05, for groups of many query vectors.
//
// A CTA takes up to 256 query vectors of one group and KV head, 128 a softmax warpgroup, and streams its share
// of the prefix 64 tokens (4 blocks) at a time; of 128 vectors:
//   S (128 x 64, tensor memory) = Q (fp16, shared memory) . K^T (codes converted to fp16, shared memory)
//   P = exp2(S * s_k * scale - m), one thread per query vector, fp16 weights P * s_v back to tensor memory
//   O (128 x 128, tensor memory) += P . V (codes converted to fp16, shared memory)
// Each block is converted once for 128 vectors; on mma.sync every 16 vectors
// convert it again, and that conversion is what bounds the 16-vector tiles.
//
// A unit is up to 256 query vectors of a group and KV head.  With more than 128 of
// them two softmax warpgroups take 128 each and meet every tile; with fewer both
// hold the same vectors and take the tiles in turn, each with its own running maximum,
// sum and O, and leave two records.
//
// Roles (512 threads, one CTA per SM): warpgroups 0 and 1 softmax (thread v = vector v =
// tensor-memory lane v), warpgroup 2 converts (warp w = block w of the 64 tokens, the next tile's codes
// already in registers), warp 12 issues the products.  Tiles pass through a ring of 4
// stages (codes as fp16, scales); S is double-buffered per softmax warpgroup and P overwrites its S.
// The registers go where the scores are: 160 a softmax thread, 112 a converting one, 80 the rest.
// (Measured before: the same products issued by softmax threads between their steps, two CTAs of
// 256 threads per SM: 75 us for 64 sequences on 32768 tokens, each issue holding its warp for 1000 cycles.)
//
// Measured: 64 sequences x 32 heads on 32768 shared tokens, int8: 79 us a call, about 50 of them here (the
// products alone would take 18, 2 x 128 vectors of a tile 1024 cycles).  A tile of 256 vectors takes
// 3000 to 3600 cycles; its shared-memory traffic takes 2340 of them: the operands of the products
// 1024, the scales that every softmax thread reads, 16 bytes at 4 wavefronts, 1024, the converted
// codes 293.  Before the first tile a CTA spends 8 us on geometry, tensor memory and
// queries, behind the last one 2 us on its record.
//
// Under a key factor (TWO) the query times the factor does not fit in 11 bits: an fp16 high and low part, both
// multiplied with the same K tile.  The low part takes the second query tile, so a unit is 128
// vectors whose two warpgroups take turns: 33 sequences of 8176 tokens, int4: 55 us a call, 50 with one part.  A group's
// last unit costs a whole pass over the prefix however few its vectors: those 33 sequences are 128 + 4 vectors a KV head,
// 2048 tile steps where 128 vectors would take 1024.
//
// Orders inside a tile.  The tokens and dims of a block are permuted so that a lane's codes
// (fragment-native order, include/kvq.h) go to shared memory as 16-byte (K) and
// 8-byte (V) stores without bank conflicts:
//   token i of block b:  column 8 b + 32 (t >> 1) + 4 (t & 1) + j,  t = (i & 7) >> 1, j = 2 (i & 1) + (i >> 3)
//   dim 32 t + 8 i + e:  half i >> 1, 16-byte chunk (t & 1) + 4 (t >> 1) + 2 (i & 1), element e
// (the same dim order for Q and K; the same token order for the columns of S and the k-index of P . V).
//
// Sequences stand apart: sigma is each vector's own, from the value scales that it sees, and a token whose scale
// is not finite counts in the rows that see it alone.  (The same calls with one sigma a warp: 3 documents
// 76.2 us for 76.6, 64 of 32768 79.5 for 79.6.  Told by the converting warps, tile by tile: 79 us for 3 documents.
// Rows that have ended have no say: with 5 empty sequences among 40 on 8192 tokens 41.3 us, 48.7 where they had.)
//
// Precision as in the decode kernel: exact codes, the query exact in fp16 (bf16 has 8 bits; or
// int8 codes, or two parts), scales in fp32, fp16 weights kept in range by the sigma offset
// (kvq_decode_impl.cuh), fp32 sums of the unrounded weights.  The weight's one rounding to fp16 (2^-11 of it at most) is
// what the outputs differ by from the formula in float32: 2.0e-4 of their norm (4 of 2048 to 64 of 32768 tokens, int8
// and int4), an eighth of what rounding the outputs to bf16 takes (1.6e-3); q_bits 32 carries the weights in two parts.
#include "kvq_shared.cuh"
#include "kvq_tc_tiles.cuh"

namespace kvq {
namespace {

struct TcSmem {
  alignas(1024) uint8_t q[2][2][kQ * 128];  // [warpgroup][half]
  alignas(1024) TcStage st[kRing];
  float sk[kRing][kTok], sv[kRing][kTok], mk[kRing][kTok], mv[kRing][kTok];
  float svmax[kRing][4];
  float qs[2 * kQ], qz[2 * kQ];
  int qlen[2 * kQ];
  // full: a stage's 128 converting threads; empty: its products are done; q_full: the softmax threads have
  // staged a segment's queries; s_full, p_full, o_done [warpgroup][S buffer]: scores, weights, P . V done
  uint64_t full[kRing], empty[kRing], q_full, seg_done, s_full[2][2], p_full[2][2], o_done[2][2];
  uint32_t tmem;
  int minlen[2];
  SharedGeo geo;
};

// The segments of a CTA, walked alike by every role: tiles t0 .. t0 + nt - 1 of a unit.
struct Segment {
  SharedUnit un;
  int nt, t0, nblk, first, rows;
  int nv;     // query vectors of the unit's tile
  bool both;  // more than 128: both warpgroups meet every tile
};
__device__ __forceinline__ Segment segment_at(const SharedGeo* geo, const DecodeArgs& a, int unit, long long x, long long x1) {
  Segment g;
  g.un = unit_at(geo, a.num_groups, a.c.H, kTok / kBlock, x);
  g.nt = int(min(x1, g.un.start + g.un.steps) - x);
  g.t0 = int(x - g.un.start);
  g.nblk = geo->g.blocks[g.un.group];
  g.first = geo->g.start[g.un.group];
  g.rows = geo->g.start[g.un.group + 1] - g.first;
  g.nv = min(g.rows * a.G - g.un.tile * unit, unit);
  g.both = g.nv > kQ;
  return g;
}
// Tiles of a segment that warpgroup j takes.
__device__ __forceinline__ int jobs_of(const Segment& g, int j) { return g.both ? g.nt : (g.nt + 1 - j) / 2; }

// TWO: queries as an fp16 high and low part, the low ones in the second query tile; units of 128 vectors.
template <int KB, int VB, bool ASYM, bool TWO>
__global__ void __launch_bounds__(kTcThreads, 1) shared_tc_kernel(const SharedArgs sa) {
  using F = Fmt<KB, VB, ASYM>;
  constexpr int kUnit = TWO ? kQ : 2 * kQ;
  constexpr int kStep = kTok / kBlock;
  constexpr float kKC = KB == 8 ? 128.f : (KB == 4 ? 8.f : 2.f), kVC = VB == 8 ? 128.f : (VB == 4 ? 8.f : 2.f);
  const DecodeArgs& a = sa.d;
  extern __shared__ uint8_t raw_smem[];
  TcSmem* sm = reinterpret_cast<TcSmem*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm->full[i], 128);
      mbar_init(&sm->empty[i], 1);
    }
    mbar_init(&sm->q_full, 2 * kQ);
    mbar_init(&sm->seg_done, 2 * kQ);
    for (int j = 0; j < 2; ++j)
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm->s_full[j][i], 1);
        mbar_init(&sm->p_full[j][i], kQ);
        mbar_init(&sm->o_done[j][i], 1);
      }
    fence_mbar_init();
  }
  // Beside the suffix kernel, see kvq_shared.cuh: the wait for it comes last.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  shared_geometry(&sm->geo, a, kUnit, kStep, tid, kTcThreads, false);  // errors are reported by the suffix kernel
  const SharedGeo* geo = &sm->geo;
  const int Pe = shared_ctas(geo, sa.sl.ctas), ci = blockIdx.x;
  if (ci >= Pe) return wait_for_suffix();
  const long long x0 = (long long)ci * geo->T / Pe, x1 = (long long)(ci + 1) * geo->T / Pe;
  if (x0 >= x1) return wait_for_suffix();
  if (warp == 12) tmem_alloc(&sm->tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, sm->tmem, 0);
  // Every wait is bounded; a role that gives up leaves its loop, the others follow when their own waits run out.
  bool ok = true;
  auto ring_wait = [&](uint64_t* bars, int n) { return mbar_wait(&bars[n & (kRing - 1)], uint32_t(n / kRing) & 1u); };
  auto pair_wait = [&](uint64_t* bars, int c) { return mbar_wait(&bars[c & 1], uint32_t(c >> 1) & 1u); };

  if (warp >= 12) {
    // ---------------------------------------------------------------- products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 12) {
      const bool leader = elect_one();
      const uint32_t q_addr = smem_u32(sm->q), st_addr = smem_u32(sm->st);
      int n0 = 0, c0 = 0, c1 = 0, seg = 0;  // tiles and jobs before this segment
      for (long long x = x0; x < x1 && ok; ++seg) {
        const Segment g = segment_at(geo, a, kUnit, x, x1);
        x += g.nt;
        ok = mbar_wait(&sm->q_full, uint32_t(seg) & 1u);
        // P . V runs one tile behind the scores, two where the warpgroups take turns
        const int lag = g.both ? 1 : 2;
        for (int i = 0; i < g.nt + lag && ok; ++i) {
          if (i < g.nt) {
            const int n = n0 + i;
            ok = ring_wait(sm->full, n);
            tc_fence_after();
            const uint64_t kd = tile_desc(st_addr + uint32_t(n & (kRing - 1)) * uint32_t(sizeof(TcStage)));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (!g.both && (i & 1) != j) continue;
              const int c = (j ? c1 : c0) + (g.both ? i : i >> 1);
              if (c >= 2) ok = ok && pair_wait(sm->o_done[j], c - 2);  // S's buffer: its weights have been read
              if (!ok) break;
              tc_fence_after();
              const uint64_t qd = tile_desc(q_addr + (g.both ? j : 0) * uint32_t(sizeof(sm->q[0])));
              const uint32_t d = tmem + 256 + 128 * j + 64 * (c & 1);
              if (leader) {
#pragma unroll
                for (int k = 0; k < kHeadDim / 16; ++k)
                  tc_mma_ss(d, qd + (k >> 2) * (sizeof(sm->q[0][0]) >> 4) + 2 * (k & 3),
                            kd + (k >> 2) * (sizeof(sm->st[0].k[0]) >> 4) + 2 * (k & 3), f16_idesc(kQ, kTok), k > 0);
                if constexpr (TWO) {
#pragma unroll
                  for (int k = 0; k < kHeadDim / 16; ++k)
                    tc_mma_ss(d, qd + (sizeof(sm->q[0]) >> 4) + (k >> 2) * (sizeof(sm->q[0][0]) >> 4) + 2 * (k & 3),
                              kd + (k >> 2) * (sizeof(sm->st[0].k[0]) >> 4) + 2 * (k & 3), f16_idesc(kQ, kTok), true);
                }
                tc_commit(&sm->s_full[j][c & 1]);
              }
              __syncwarp();
            }
          }
          const int p = i - lag;
          if (p >= 0 && ok) {
            const int n = n0 + p, s = n & (kRing - 1);
            const uint64_t vd = tile_desc(st_addr + uint32_t(s) * uint32_t(sizeof(TcStage)) + uint32_t(sizeof(sm->st[0].k)));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (!g.both && (p & 1) != j) continue;
              const int job = g.both ? p : p >> 1, c = (j ? c1 : c0) + job;
              ok = ok && pair_wait(sm->p_full[j], c);
              if (!ok) break;
              tc_fence_after();
              const uint32_t d = tmem + 128 * j, w = tmem + 256 + 128 * j + 64 * (c & 1);
              if (leader) {
#pragma unroll
                for (int k = 0; k < kTok / 16; ++k)
                  tc_mma_ts(d, w + 8 * k, vd + 2 * k, f16_idesc(kQ, kHeadDim), job > 0 || k > 0);
                tc_commit(&sm->o_done[j][c & 1]);
                if (j == 1 || !g.both) tc_commit(&sm->empty[s]);
              }
              __syncwarp();
            }
          }
        }
        n0 += g.nt;
        c0 += jobs_of(g, 0);
        c1 += jobs_of(g, 1);
      }
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- conversion
    asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    const int w = warp - 8;
    const uint32_t km = magic_f16x2(a.B);
    const uint32_t c64 = 0x64646464u | (uint32_t(a.B) >> 16);  // a.B <= 4096: the constant itself
    int n = 0;
    for (long long x = x0; x < x1 && ok;) {
      const Segment g = segment_at(geo, a, kUnit, x, x1);
      x += g.nt;
      const int* table = a.table + size_t(g.first) * a.mbps;
      int ids = -1, ids_next = -1;  // this warp's table entries of 32 tiles, and of the next 32
      auto load_ids = [&](int i) {
        const int blk = (g.t0 + i + lane) * kStep + w;
        int id = -1;
        if (i + lane < g.nt && blk < g.nblk) {
          id = __ldcg(table + blk);
          if (id < 0 || id >= a.c.num_blocks) {
            flag(a.err, KVQ_DEVERR_BLOCK_ID);
            id = 0;
          }
        }
        return id;
      };
      ids_next = load_ids(0);
      int maxlen = 0;  // of the unit's rows: scales of slots behind it are not data
      for (int r = g.un.tile * kUnit / a.G + lane; r <= (g.un.tile * kUnit + g.nv - 1) / a.G; r += 32)
        maxlen = max(maxlen, prefix_len(a, g.first + r, g.nblk));
      maxlen = __reduce_max_sync(kFull, maxlen);
      // this warp's block of the tile: codes, and the record entries of token `lane` (lanes 0..15)
      Raw<KB> rk;
      Raw<VB> rv;
      float ks = 0.f, vs = 0.f, ko = 0.f, vo = 0.f;
      auto block_of = [&](int i) {  // called once per tile, in order
        if ((i & 31) == 0) {
          ids = ids_next;
          ids_next = load_ids(i + 32);
        }
        return i < g.nt ? __shfl_sync(kFull, ids, i & 31) : -1;
      };
      auto fetch_keys = [&](int phys) {
        ks = vs = ko = vo = 0.f;
        rk.clear();
        if (phys < 0) return;
        const size_t hb = size_t(g.un.h) * a.c.num_blocks + phys;
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
        if (phys >= 0) rv.load(a.c.v_codes + (size_t(g.un.h) * a.c.num_blocks + phys) * F::kVBB, lane);
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
        const bool data = ((g.t0 + i) * kStep + w) * kBlock + lane < maxlen;
        if (!data) vs = 0.f;
        if (lane < kBlock) {
          const int col = tile_col(w, lane);
          sm->sk[s][col] = ks;
          sm->sv[s][col] = vs;
          if constexpr (ASYM) {
            sm->mk[s][col] = fmaf(kKC, ks, ko);
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
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    const int j = warp >> 2, v = tid & (kQ - 1);  // warpgroup, its vector
    const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t o_cols = lanes + 128 * j, s_cols = lanes + 256 + 128 * j;
    int n0 = 0, c = 0, c_other = 0, seg = 0;  // tiles before this segment; this warpgroup's and the other's jobs so far
    for (long long x = x0; x < x1 && ok; ++seg) {
      const Segment g = segment_at(geo, a, kUnit, x, x1);
      x += g.nt;
      if (seg > 0) {  // both warpgroups are done with the previous segment's queries
        mbar_arrive(&sm->seg_done);
        ok = __all_sync(kFull, mbar_wait(&sm->seg_done, uint32_t(seg - 1) & 1u));
        if (!ok) break;
      }
      {
        // this warp's 32 vectors (16 of the shared 128), 4 a step
        const int per = g.both ? 32 : 16, v0 = (g.both ? warp : 2 * (warp & 3) + j) * per, sub = lane & 7;
        const int G = a.G, gv0 = g.un.tile * kUnit + v0;
        const uint16_t* src = a.q + (size_t(g.first) * a.Hq + g.un.h * G) * kHeadDim + 16 * sub;
        float f[16];
        if (a.c.factor) {
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<float4*>(f + k) =
                __ldcg(reinterpret_cast<const float4*>(a.c.factor + g.un.h * kHeadDim + 16 * sub + k));
        }
        uint8_t* half = sm->q[g.both ? j : 0][sub & 1];
        int r = (gv0 + (lane >> 3)) / G, hj = (gv0 + (lane >> 3)) % G;
        uint4 raw[8][2];  // all loads before the first conversion: one latency
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
          if (4 * i < per && r < g.rows) {
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
          const int row = (gv0 + lane) / G;
          sm->qlen[v0 + lane] = row < g.rows ? prefix_len(a, g.first + row, g.nblk) : 0;
        }
#pragma unroll 1
        for (int b = 0; b < per; b += 4) {
          const uint4 cur[2] = {raw[0][0], raw[0][1]};
#pragma unroll
          for (int e = 0; e < 7; ++e) {  // rotate: the loop stays short and every index is known
            raw[e][0] = raw[e + 1][0];
            raw[e][1] = raw[e + 1][1];
          }
          const int at = v0 + b + (lane >> 3);
          float qs, sum;
          put_query<ASYM, TWO>(a, cur, f, half, int(sizeof(sm->q[0])), at & (kQ - 1), sub, qs, sum);
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
      const int at = g.both ? tid : v;
      const float qs = sm->qs[at], qz = ASYM ? sm->qz[at] : 0.f;
      const int len = sm->qlen[at];
      // the warp's shortest row decides whether a tile needs the mask at all (unused vectors do not count)
      const int minlen = __reduce_min_sync(kFull, at < g.nv ? len : 0x7fffffff);
      float m = kNegInf, l = 0.f, z = 0.f, sg = float(kSigma0);
      float svlim = ldexpf(1.f, kWeightExp - int(kMaxSlack) - kSigma0);
      const int jobs = jobs_of(g, j);
#pragma unroll 1
      for (int i = 0; i < jobs; ++i, ++c) {
        const int tile = g.both ? i : 2 * i + j, sc = (n0 + tile) & (kRing - 1);
        ok = __all_sync(kFull, ring_wait(sm->full, n0 + tile) && pair_wait(sm->s_full[j], c));  // scales, scores
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = s_cols + 64 * (c & 1);
        uint32_t r[kTok];
        tmem_ld32(st, r);
        tmem_ld32(st + 32, r + 32);
        tc_wait_ld();
        const int tok0 = (g.t0 + tile) * kTok;
#pragma unroll
        for (int k = 0; k < kTok; k += 4) {
          const float4 ks = *reinterpret_cast<const float4*>(&sm->sk[sc][k]);
          if constexpr (ASYM) {
            const float4 ko = *reinterpret_cast<const float4*>(&sm->mk[sc][k]);
            fma2(r[k], r[k + 1], ks.x, ks.y, ko.x * qz, ko.y * qz);
            fma2(r[k + 2], r[k + 3], ks.z, ks.w, ko.z * qz, ko.w * qz);
          } else {
            mul2(r[k], r[k + 1], ks.x, ks.y);
            mul2(r[k + 2], r[k + 3], ks.z, ks.w);
          }
        }
        if (tok0 + kTok > minlen) {  // a row of the warp ends inside this tile or before it
#pragma unroll
          for (int k = 0; k < kTok; ++k)
            if (tok0 + tile_token(k) >= len) r[k] = __float_as_uint(kNegInf);
        }
        float x4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
        for (int k = 0; k < kTok; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x4[e] = fmaxf(x4[e], fmaxf(__uint_as_float(r[k + 2 * e]), __uint_as_float(r[k + 2 * e + 1])));
        const float mx = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * qs;
        const float4 sm4 = *reinterpret_cast<const float4*>(sm->svmax[sc]);
        const float svm = max_nan(max_nan(sm4.x, sm4.y), max_nan(sm4.z, sm4.w));  // the same in every thread
        if (__any_sync(kFull, mx > m + kMaxSlack || !(svm <= svlim))) {
          float f = 1.f;
          if (__any_sync(kFull, mx > m + kMaxSlack)) {
            const float mn = fmaxf(m, mx);
            f = mn == kNegInf ? 1.f : ex2(m - mn);
            m = mn;
          }
          float sv = svm;
          if (!(svm <= kFloatMax)) {
            // A value scale that is not finite: -1 stands for it, as in rows that do not see its token 0 x inf would be
            // no number.  Every warp that goes on to use the scales writes the same.
            for (int k = lane; k < kTok; k += 32)
              if (!(fabsf(sm->sv[sc][k]) <= kFloatMax)) {
                sm->sv[sc][k] = -1.f;
                if constexpr (ASYM) sm->mv[sc][k] = 0.f;
              }
            __syncwarp();
          }
          // by the scales that this row sees: a token leaves other sequences alone
          if (len <= tok0) {  // the row has ended, or was never there
            sv = 0.f;
            svlim = fmaxf(svlim, kFloatMax);
          } else if (!(svm <= svlim) && (len < tok0 + kTok || !(svm <= kFloatMax))) {
            float least = 0.f;
            sv = 0.f;
#pragma unroll 1
            for (int k = 0; k < kTok; ++k) {
              const float own = tok0 + tile_token(k) < len ? sm->sv[sc][k] : 0.f;
              sv = fmaxf(sv, own);
              least = fminf(least, own);
            }
            if (least < 0.f) svlim = -kNegInf;  // the row's outputs are no numbers
          }
          if (sv > svlim) {
            int e;
            frexpf(sv, &e);
            const int sn = min(int(sg), kWeightExp - int(kMaxSlack) - e);
            f *= ldexpf(1.f, sn - int(sg));
            sg = float(sn);
            svlim = ldexpf(1.f, kWeightExp - int(kMaxSlack) - sn);
          }
          l *= f;
          z *= f;
          if (i > 0) {  // O too, once the products so far are complete
            ok = __all_sync(kFull, pair_wait(sm->o_done[j], c - 1));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < kHeadDim; k += 32) {
              uint32_t o[32];
              tmem_ld32(o_cols + k, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(o_cols + k, o);
            }
            tc_wait_st();
          }
        }
        const float base = m == kNegInf ? 0.f : m - sg;
        uint32_t la[4] = {0u, 0u, 0u, 0u};  // four partial sums of the weights
#pragma unroll
        for (int half = 0; half < kTok; half += 32) {
          uint32_t p[16];
#pragma unroll
          for (int k = half; k < half + 32; k += 4) {
            const float4 vs = *reinterpret_cast<const float4*>(&sm->sv[sc][k]);
            fma2(r[k], r[k + 1], qs, qs, -base, -base);
            fma2(r[k + 2], r[k + 3], qs, qs, -base, -base);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[k + e] = __float_as_uint(ex2(__uint_as_float(r[k + e])));
            add2(la[0], la[1], r[k], r[k + 1]);
            add2(la[2], la[3], r[k + 2], r[k + 3]);
            if constexpr (ASYM) {
              const float4 vo = *reinterpret_cast<const float4*>(&sm->mv[sc][k]);
              z = fmaf(__uint_as_float(r[k]), vo.x, fmaf(__uint_as_float(r[k + 1]), vo.y, z));
              z = fmaf(__uint_as_float(r[k + 2]), vo.z, fmaf(__uint_as_float(r[k + 3]), vo.w, z));
            }
            mul2(r[k], r[k + 1], vs.x, vs.y);
            mul2(r[k + 2], r[k + 3], vs.z, vs.w);
            p[(k - half) / 2] = pack_half2(__uint_as_float(r[k]), __uint_as_float(r[k + 1]));
            p[(k - half) / 2 + 1] = pack_half2(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3]));
          }
          tmem_st16(st + half / 2, p);  // over S, which has been read
        }
        l += (__uint_as_float(la[0]) + __uint_as_float(la[1])) + (__uint_as_float(la[2]) + __uint_as_float(la[3]));
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&sm->p_full[j][c & 1]);
      }
      if (!ok) break;
      // ---- this segment's record: vectors 128 j .. of the unit, or the second record of its 128 vectors
      if (jobs > 0) {
        ok = __all_sync(kFull, pair_wait(sm->o_done[j], c - 1));
        if (!ok) break;
        tc_fence_after();
      }
      if constexpr (TWO) {  // the other warpgroup's scores have read the low query parts, whose place the records pass by
        const int others = jobs_of(g, 1 - j);
        c_other += others;
        if (others > 0) ok = __all_sync(kFull, pair_wait(sm->s_full[1 - j], c_other - 1));
        if (!ok) break;
      }
      if (g.both ? tid < g.nv : v < g.nv) {
        const size_t slot = size_t(ci + g.un.u) * 2 * kQ + tid;
        reinterpret_cast<float*>(a.ws + sa.sl.off_m)[slot] = m == kNegInf ? kNegInf : m - sg;
        reinterpret_cast<float*>(a.ws + sa.sl.off_l)[slot] = l;
      }
      const int used = min(32, (g.both ? g.nv - j * kQ : g.nv) - (warp & 3) * 32);  // this warp's vectors in use
      if (jobs > 0 && used > 0) {
        // O's rows to global memory as whole 128-byte lines, by way of 4 KB of this warp's in a part of Q
        // that no product reads any more (its own Q; the unused second one where both share the first)
        float4* buf = reinterpret_cast<float4*>(g.both ? sm->q[j][0] : sm->q[1][j]) + (warp & 3) * 256;
        const float add = svlim == -kNegInf ? __int_as_float(0x7fffffff) : z;
        float4* rec = reinterpret_cast<float4*>(a.ws + sa.sl.off_rec) +
                      (size_t(ci + g.un.u) * 2 * kQ + warp * 32) * (kHeadDim / 4);
#pragma unroll 1
        for (int k = 0; k < kHeadDim; k += 32) {
          uint32_t o[32];
          tmem_ld32(o_cols + k, o);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            buf[lane * 8 + (e ^ (lane & 7))] =
                make_float4(__uint_as_float(o[4 * e]) + add, __uint_as_float(o[4 * e + 1]) + add,
                            __uint_as_float(o[4 * e + 2]) + add, __uint_as_float(o[4 * e + 3]) + add);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int row = 4 * e + (lane >> 3);
            if (row < used) rec[size_t(row) * (kHeadDim / 4) + k / 4 + (lane & 7)] = buf[row * 8 + ((lane & 7) ^ (row & 7))];
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      n0 += g.nt;
    }
  }
  if (!ok) flag(a.err, KVQ_DEVERR_TIMEOUT);
  wait_for_suffix();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_free(tmem, kTmemCols);
}

template <int KB, int VB, bool ASYM, bool TWO>
struct SharedTcKernel {
  static int smem_bytes() { return int(sizeof(TcSmem)) + 1024; }
  // CTAs of one wave on the current device.
  static int ctas() {
    static std::mutex mu;
    static std::map<int, int> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lk(mu);
    auto it = done.find(dev);
    if (it != done.end()) return it->second;
    int sms = 0;
    const auto k = shared_tc_kernel<KB, VB, ASYM, TWO>;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes()) != cudaSuccess ||
        cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess)
      return 0;
    return done[dev] = sms;  // one CTA per SM: its shared memory and all of its tensor memory
  }
  static cudaError_t launch(const SharedArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.sl.ctas));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = smem_bytes();
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, shared_tc_kernel<KB, VB, ASYM, TWO>, a);
  }
};

template <bool TWO, class F>
auto by_format_two(const CacheView& c, F f) {
  const int kb = c.k_bits, vb = c.v_bits;
  const bool as = c.asym != 0;
  if (kb == 8 && vb == 8) return as ? f(SharedTcKernel<8, 8, true, TWO>{}) : f(SharedTcKernel<8, 8, false, TWO>{});
  if (kb == 4 && vb == 4) return as ? f(SharedTcKernel<4, 4, true, TWO>{}) : f(SharedTcKernel<4, 4, false, TWO>{});
  if (kb == 4 && vb == 8) return as ? f(SharedTcKernel<4, 8, true, TWO>{}) : f(SharedTcKernel<4, 8, false, TWO>{});
  if (kb == 8 && vb == 4) return as ? f(SharedTcKernel<8, 4, true, TWO>{}) : f(SharedTcKernel<8, 4, false, TWO>{});
  return as ? f(SharedTcKernel<2, 2, true, TWO>{}) : f(SharedTcKernel<2, 2, false, TWO>{});
}

template <class F>
auto by_format(const CacheView& c, F f) {
  return c.q_bits == 32 ? by_format_two<true>(c, f) : by_format_two<false>(c, f);
}

}  // namespace

int shared_tc_ctas(const CacheView& c) {
  return by_format(c, [](auto k) { return decltype(k)::ctas(); });
}

cudaError_t launch_shared_tc(const SharedArgs& a, cudaStream_t s) {
  return by_format(a.d.c, [&](auto k) { return decltype(k)::launch(a, s); });
}

}  // namespace kvq
