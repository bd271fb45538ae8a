// The tokens behind the shared prefixes (kvq_decode_shared): decode attention of
// every (sequence, KV head) over its own blocks, one record (m, l, o) per chunk.
//
// The suffixes are short and many, and a merge follows in any case, so the work
// is cut into chunks of whole (sequence, KV head) units or parts of them: a chunk
// has C blocks, C from the total number of blocks and the CTAs (about one chunk for
// two of them), so that one long suffix among short ones is shared out too.  There are no
// tickets and no waiting: chunk k writes record k.  (The Stream-K decode
// kernel over the same tokens spends about 8 us per unit start on its flush, ticket and
// merge: 34 us for 64 x 8 suffixes of 500 tokens that take 10 us to read.)  Here they take 20 (27 from a cold L2,
// 72 MB), bound by latency: a chunk is three steps a warp, behind the lengths, the groups, the table and the queries, each a
// load that waits for the one before.
//
// A warp streams its blocks through its own shared-memory stages with 16-byte
// asynchronous copies (each lane copies the pieces it will read) and runs the decode
// kernel's block routine on them.  The bf16 window of a unit is a chunk of its own.
#pragma once

#include "kvq_shared.cuh"

namespace kvq {
namespace {

constexpr int kSufThreads = kConsumers;  // 4 warps, the decode kernel's consumers
constexpr int kSufMinGroups = 2;         // a chunk has at least this many block groups per warp

template <int KB, int VB, bool ASYM>
struct SufFmt {
  using F = Fmt<KB, VB, ASYM>;
  static constexpr int kNB = F::kBPW;  // blocks a warp takes together
  static constexpr int kStage = kNB * F::kPerBlock;
  static constexpr int kStages = KB == 16 ? 2 : (KB == 8 && VB == 8 ? 2 : 3);
  static constexpr int kRing = kStages * kStage;  // of one warp
  static constexpr int kOffV = kNB * F::kKBB, kOffMeta = kOffV + kNB * F::kVBB;
};

// Shared-memory map behind the rings (16-byte aligned offsets).
struct SufSmem {
  int merge_o, merge_ml, qh, qlo, qs, nblk, lens, groups, total;
};
__host__ __device__ inline SufSmem suf_smem(int rings, int B, bool loq) {
  SufSmem m;
  int o = rings;
  m.merge_o = o;  o += kConsumerWarps * 4 * kHeadDim * 4;
  m.merge_ml = o; o += 2 * kConsumerWarps * kMaxGroup * 4;
  m.qh = o;       o += kMaxGroup * kHeadDim * 2;
  m.qlo = o;      o += loq ? kMaxGroup * kHeadDim * 2 : 0;
  m.qs = o;       o += 4 * kMaxGroup * 4;
  m.nblk = o;     o += ((B + 1) * 4 + 15) / 16 * 16;  // chunks of one head before sequence b
  m.lens = o;     o += (B * 4 + 15) / 16 * 16;
  m.groups = o;   o += (int(sizeof(GroupGeo)) + 15) / 16 * 16;
  m.total = o;
  return m;
}

// Sequence b of length L: its prefix's blocks, tokens behind it (stored ones) and ring tokens.
struct SufLen {
  int skip, tokens, ring;
};
__device__ __forceinline__ SufLen suffix_len(const DecodeArgs& a, const GroupGeo* groups, int b, int L, bool& bad) {
  const int W = a.c.window, cap = table_tokens(a.mbps, W);
  if (L < 0 || L > cap) {
    bad = true;
    L = min(max(L, 0), cap);
  }
  const int g = group_of(groups, a.num_groups, b), stored = max(L - W, 0);
  SufLen s;
  s.skip = g < 0 ? 0 : groups->blocks[g];
  s.tokens = max(stored - s.skip * kBlock, 0);
  s.ring = min(L, W);
  return s;
}

// The query group's rows as B operands, as write_query_rows lays them out: 8 lanes a
// row (16 dims each, their bf16 bits in raw), all rows in one step by warps 0 and 1.
template <bool kBf16, bool ASYM, bool LOQ>
__device__ __forceinline__ void put_rows(const DecodeArgs& a, const uint4 (&raw)[2], int h, uint16_t* qh, uint32_t* qlo,
                                         float* qs, int tid) {
  if (tid >= 8 * kMaxGroup) return;
  const int q = tid >> 3, sub = tid & 7;
  float f[16];
  uint4* row = reinterpret_cast<uint4*>(qh + q * kHeadDim + 16 * sub);
  if constexpr (kBf16) {
    row[0] = raw[0];
    row[1] = raw[1];
    if (sub == 0) qs[q] = kLog2e * kInvSqrtD;
    return;
  }
  if (a.c.factor) {
#pragma unroll
    for (int k = 0; k < 16; k += 4)
      *reinterpret_cast<float4*>(f + k) = *reinterpret_cast<const float4*>(a.c.factor + h * kHeadDim + 16 * sub + k);
  }
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 4 ? (&raw[0].x)[i] : (&raw[1].x)[i - 4];
    x[2 * i] = __uint_as_float(w << 16);
    x[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
  }
  if (a.c.factor) {
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] *= f[k];
  }
  float am = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) am = fmaxf(am, fabsf(x[k]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(kFull, am, o));
  float scale = kLog2e * kInvSqrtD;
  if (a.c.q_bits == 8) {
    float s = 1.f;
#pragma unroll 1
    for (int k = 0; k < 16; k += 4) {  // a loop: the rounding with its exact ties is long code
      const float y[4] = {x[0], x[1], x[2], x[3]};
      float c[4];
      s = quantize_int8_row(y, am, c);
#pragma unroll
      for (int e = 0; e < 12; ++e) x[e] = x[e + 4];  // rotate, so that every index is known
#pragma unroll
      for (int e = 0; e < 4; ++e) x[12 + e] = c[e];
    }
    scale *= s;
  } else {
    // exact powers of two: am * 2^(14 - e) in [2^14, 2^15); below 2^-112 the scores are zero to any precision
    const uint32_t e = max(__float_as_uint(am) >> 23, 15u);
    const float f2 = __uint_as_float((268u - e) << 23);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] *= f2;
    scale *= __uint_as_float((e - 14u) << 23);
  }
  float even = 0.f, odd = 0.f, z = 0.f;  // sums of the row as the MMA sees it: by k-slice, with the low parts
  uint32_t hi[8], lo[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = pack_half2(x[2 * i], x[2 * i + 1]);
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi[i]));
    if (i & 2) odd += y.x + y.y;
    else even += y.x + y.y;
    if constexpr (LOQ) {
      lo[i] = pack_half2(x[2 * i] - y.x, x[2 * i + 1] - y.y);
      const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&lo[i]));
      z += w.x + w.y;
    }
  }
  row[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  row[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
  if constexpr (LOQ) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4*>(qlo + ((2 * (sub & 1) + i) * 32 + 4 * q + (sub >> 1)) * 4) =
          make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    even += __shfl_xor_sync(kFull, even, o);
    odd += __shfl_xor_sync(kFull, odd, o);
    if constexpr (ASYM && LOQ) z += __shfl_xor_sync(kFull, z, o);
  }
  if (sub == 0) {
    qs[q] = scale;
    if constexpr (ASYM) qs[kMaxGroup + q] = even + odd + z;
    qs[2 * kMaxGroup + (q >> 1) * 4 + (q & 1)] = -kOffsetF16 * even;
    qs[2 * kMaxGroup + (q >> 1) * 4 + 2 + (q & 1)] = -kOffsetF16 * odd;
  }
}

template <int KB, int VB, bool ASYM, bool LOQ>
__global__ void __launch_bounds__(kSufThreads, 4) suffix_kernel(const SharedArgs sa) {
  using F = Fmt<KB, VB, ASYM>;
  using T = SufFmt<KB, VB, ASYM>;
  constexpr int NB = T::kNB, S = T::kStages;
  const DecodeArgs& a = sa.d;
  extern __shared__ __align__(128) uint8_t smem[];
  const SufSmem mp = suf_smem(kConsumerWarps * T::kRing, a.B, LOQ);
  float* merge_o = reinterpret_cast<float*>(smem + mp.merge_o);
  float* merge_m = reinterpret_cast<float*>(smem + mp.merge_ml);
  float* merge_l = merge_m + kConsumerWarps * kMaxGroup;
  uint16_t* qh = reinterpret_cast<uint16_t*>(smem + mp.qh);
  uint32_t* qlo_s = reinterpret_cast<uint32_t*>(smem + mp.qlo);
  float* qs = reinterpret_cast<float*>(smem + mp.qs);
  int* pre = reinterpret_cast<int*>(smem + mp.nblk);
  int* lens = reinterpret_cast<int*>(smem + mp.lens);
  GroupGeo* groups = reinterpret_cast<GroupGeo*>(smem + mp.groups);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = a.B, H = a.c.H, G = a.G, W = a.c.window;
  uint8_t* const ring = smem + warp * T::kRing;
  if constexpr (!F::kBf16) {
    // keys under per-channel scales only: the key-scale slots hold 1.0 (never copied over)
    if (a.c.k_chan)
      for (int i = lane; i < S * NB * kBlock; i += 32)
        reinterpret_cast<float*>(ring + (i / (NB * kBlock)) * T::kStage + T::kOffMeta)[(i / kBlock % NB) * F::kMF + F::kKS +
                                                                                      i % kBlock] = 1.f;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the prefix kernel may start: it reads nothing that is not complete by now
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the first lengths beside the groups: every load that waits for another one costs its latency
  const int len0 = tid < B ? a.seq_lens[tid] : 0;
  const unsigned gbad = load_groups(groups, a.group_start, a.prefix_blocks, a.num_groups, B, a.mbps, tid, kSufThreads);
  if (gbad && blockIdx.x == 0 && tid == 0) flag(a.err, gbad);

  // ---- chunks: C blocks each, of all units in (sequence, head, block) order
  bool bad = false;
  int mine = 0;
  for (int b = tid; b < B; b += kSufThreads) {
    const int L = b == tid ? len0 : a.seq_lens[b];
    const int n = (suffix_len(a, groups, b, L, bad).tokens + kBlock - 1) / kBlock;
    lens[b] = L;
    pre[b + 1] = n;
    mine += n;
  }
  if (bad && blockIdx.x == 0) flag(a.err, KVQ_DEVERR_SEQ_LEN);
  if (tid == 0) pre[0] = 0;
  mine = __reduce_add_sync(kFull, mine);
  if (lane == 0) reinterpret_cast<int*>(merge_m)[warp] = mine;
  __syncthreads();
  const int* part = reinterpret_cast<const int*>(merge_m);
  const long long blocks = (long long)H * (part[0] + part[1] + part[2] + part[3]);
  constexpr int kGroup4 = kConsumerWarps * NB;
  // half a wave of chunks: fewer starts and records, and SMs that the prefix kernel can have (64 sequences of 1..1000
  // own tokens on 32768 shared ones: 80 us a call, 84 with a whole wave and 80 with a quarter)
  const long long want = (sa.sl.suf_ctas + 1) / 2;
  const int C = int(max((blocks + want - 1) / want, (long long)kSufMinGroups * kGroup4));
  __syncthreads();  // part has been read
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base < B; base += 32) {
      const int i = base + lane;
      const int own = i < B ? (pre[i + 1] + C - 1) / C : 0;
      int v = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += n;
      }
      if (i < B) {
        pre[i + 1] = v + carry;
        // for the merge: this sequence's chunks
        if (blockIdx.x == 0)
          reinterpret_cast<int2*>(a.ws + sa.sl.off_chunks)[i] = make_int2(H * (v + carry - own), own);
      }
      carry += __shfl_sync(kFull, v, 31);
    }
  }
  __syncthreads();
  const int chunks = H * pre[B], all = chunks + (W > 0 ? B * H : 0);
  const uint32_t km = magic_f16x2(B);
  float* rec_m = reinterpret_cast<float*>(a.ws + sa.sl.off_sm);
  float* rec_l = reinterpret_cast<float*>(a.ws + sa.sl.off_sl);
  float* rec_o = reinterpret_cast<float*>(a.ws + sa.sl.off_so);

  for (int k = blockIdx.x; k < all; k += gridDim.x) {
    const bool win = k >= chunks;
    int b, h, j = 0;
    if (win) {
      b = (k - chunks) / H;
      h = (k - chunks) % H;
    } else {
      int lo = 0, hi = B - 1;
      while (lo < hi) {  // the last sequence with H * pre[b] <= k that has chunks
        const int mid = (lo + hi + 1) >> 1;
        if (H * pre[mid] <= k) lo = mid;
        else hi = mid - 1;
      }
      b = lo;
      const int nc = pre[b + 1] - pre[b], i = k - H * pre[b];
      h = i / nc;
      j = i % nc;
    }
    bool ignored = false;
    const SufLen sl = suffix_len(a, groups, b, lens[b], ignored);
    const int b0 = j * C, b1 = win ? 0 : min(b0 + C, (sl.tokens + kBlock - 1) / kBlock);
    // the queries' loads first, with the table's
    uint4 raw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (!win && (tid >> 3) < G) {
      const uint4* p =
          reinterpret_cast<const uint4*>(a.q + (size_t(b) * a.Hq + h * G + (tid >> 3)) * kHeadDim + 16 * (tid & 7));
      raw[0] = p[0];
      raw[1] = p[1];
    }
    // ---- this warp's block groups: b0 + (warp + 4 i) * NB
    const int* table = a.table + size_t(b) * a.mbps + sl.skip;
    int ids = 0, ids_base = 0;
    auto load_ids = [&](int from) {  // 32 table entries of this warp: group i's block e is entry (i * NB + e)
      const int blk = b0 + ((from + lane) / NB * kConsumerWarps + warp) * NB + (from + lane) % NB;
      int v = 0;
      if (blk < b1) {
        v = table[blk];
        if (v < 0 || v >= a.c.num_blocks) {
          flag(a.err, KVQ_DEVERR_BLOCK_ID);
          v = 0;
        }
      }
      ids_base = from;
      return v;
    };
    const int groups_w = max(0, (b1 - b0 + NB - 1) / NB - warp + kConsumerWarps - 1) / kConsumerWarps;
    if (groups_w > 0) ids = load_ids(0);
    auto fetch = [&](int i) {
      if (i < groups_w) {
        if (i * NB >= ids_base + 32) ids = load_ids(i * NB);
        uint8_t* st = ring + (i % S) * T::kStage;
#pragma unroll
        for (int e = 0; e < NB; ++e) {
          if (b0 + (i * kConsumerWarps + warp) * NB + e >= b1) break;
          const int phys = __shfl_sync(kFull, ids, i * NB + e - ids_base);
          const size_t hb = size_t(h) * a.c.num_blocks + phys;
          const uint8_t* kp = a.c.k_codes + hb * F::kKBB + lane * 16;
          const uint8_t* vp = a.c.v_codes + hb * F::kVBB + lane * 16;
#pragma unroll
          for (int c = 0; c < F::kKBB / 512; ++c) cp_async16(st + e * F::kKBB + c * 512 + lane * 16, kp + c * 512);
#pragma unroll
          for (int c = 0; c < F::kVBB / 512; ++c)
            cp_async16(st + T::kOffV + e * F::kVBB + c * 512 + lane * 16, vp + c * 512);
          if constexpr (!F::kBf16) {
            const bool skip_keys = a.c.k_chan && lane * 16 < F::kVS * 4;
            if (lane < F::kMB / 16 && !skip_keys)
              cp_async16(st + T::kOffMeta + e * F::kMB + lane * 16, a.c.meta + hb * F::kMF + lane * 4);
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);

    // ---- the query group as B-operand rows
    WarpState st;
    st.reset();
    uint32_t qf[16];
    float qs0, qs1, qz0 = 0.f, qz1 = 0.f;
    __syncthreads();  // the previous chunk's queries and states have been read
    if (win) {
      stage_query<true>(a, b, h, qh, qs, warp, lane);
    } else {
      put_rows<F::kBf16, ASYM, LOQ>(a, raw, h, qh, qlo_s, qs, tid);
    }
    __syncthreads();
    load_query(qh, qs, qf, qs0, qs1, lane);
    if constexpr (ASYM) {
      qz0 = qs[kMaxGroup + 2 * (lane & 3)];
      qz1 = qs[kMaxGroup + 2 * (lane & 3) + 1];
    }
    const float4* qzo = reinterpret_cast<const float4*>(qs + 2 * kMaxGroup);
    const uint4* qlo = LOQ ? reinterpret_cast<const uint4*>(qlo_s) + lane : nullptr;

    if (win) {
      const size_t ring0 = size_t(b * H + h) * (W / kBlock);
      for (int i = warp; i * kBlock < sl.ring; i += kConsumerWarps) {
        const uint8_t* const kbs[1] = {a.c.k_win + (ring0 + i) * block_bytes(16)};
        const uint8_t* const vbs[1] = {a.c.v_win + (ring0 + i) * block_bytes(16)};
        const float* const nos[1] = {nullptr};
        const int val[1] = {min(kBlock, sl.ring - i * kBlock)};
        process_blocks<16, 16, 1, false, false>(kbs, vbs, nos, nos, nos, nos, val, qf, nullptr, nullptr, qs0, qs1, 0.f,
                                                0.f, st, lane, 0u);
      }
    }
    for (int i = 0; i < groups_w; ++i) {
      fetch(i + S - 1);
      cp_async_wait<S - 1>();
      __syncwarp();
      const uint8_t* stg = ring + (i % S) * T::kStage;
      const int blk = b0 + (i * kConsumerWarps + warp) * NB;
      auto meta = [&](int e) { return reinterpret_cast<const float*>(stg + T::kOffMeta + e * F::kMB); };
      auto ksp = [&](int e) { return F::kBf16 ? nullptr : meta(e) + F::kKS; };
      auto vsp = [&](int e) { return F::kBf16 ? nullptr : meta(e) + F::kVS; };
      auto kop = [&](int e) { return ASYM ? meta(e) + F::kKO : nullptr; };
      auto vop = [&](int e) { return ASYM ? meta(e) + F::kVO : nullptr; };
      auto val = [&](int e) { return min(kBlock, sl.tokens - (blk + e) * kBlock); };
      if (NB == 2 && blk + 1 < b1) {
        const uint8_t* const kbs[2] = {stg, stg + F::kKBB};
        const uint8_t* const vbs[2] = {stg + T::kOffV, stg + T::kOffV + F::kVBB};
        const float* const kss[2] = {ksp(0), ksp(1)};
        const float* const vss[2] = {vsp(0), vsp(1)};
        const float* const kos[2] = {kop(0), kop(1)};
        const float* const vos[2] = {vop(0), vop(1)};
        const int vals[2] = {val(0), val(1)};
        process_blocks<KB, VB, 2, ASYM, LOQ>(kbs, vbs, kss, vss, kos, vos, vals, qf, qlo, qzo, qs0, qs1, qz0, qz1, st,
                                             lane, km);
      } else {
        const uint8_t* const kbs[1] = {stg};
        const uint8_t* const vbs[1] = {stg + T::kOffV};
        const float* const kss[1] = {ksp(0)};
        const float* const vss[1] = {vsp(0)};
        const float* const kos[1] = {kop(0)};
        const float* const vos[1] = {vop(0)};
        const int vals[1] = {val(0)};
        process_blocks<KB, VB, 1, ASYM, LOQ>(kbs, vbs, kss, vss, kos, vos, vals, qf, qlo, qzo, qs0, qs1, qz0, qz1, st,
                                             lane, km);
      }
      __syncwarp();  // every lane has read the stage before it is filled again
    }

    // ---- the four warps' states into record k, four queries a pass
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      st.l0 += __shfl_xor_sync(kFull, st.l0, o);
      st.l1 += __shfl_xor_sync(kFull, st.l1, o);
    }
    if constexpr (ASYM) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        st.z0 += __shfl_xor_sync(kFull, st.z0, o);
        st.z1 += __shfl_xor_sync(kFull, st.z1, o);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        st.O[i][0] += st.z0;
        st.O[i][2] += st.z0;
        st.O[i][1] += st.z1;
        st.O[i][3] += st.z1;
      }
    }
    if (g == 0) {
      merge_m[warp * kMaxGroup + 2 * t] = st.m0 - st.sg;
      merge_m[warp * kMaxGroup + 2 * t + 1] = st.m1 - st.sg;
      merge_l[warp * kMaxGroup + 2 * t] = st.l0;
      merge_l[warp * kMaxGroup + 2 * t + 1] = st.l1;
    }
    for (int pass = 0; pass * 4 < G; ++pass) {
      if (pass > 0) __syncthreads();
      if ((t >> 1) == pass) {
        float* ow = merge_o + warp * 4 * kHeadDim;
        const int q0 = 2 * t - 4 * pass;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          ow[q0 * kHeadDim + 16 * mt + g] = st.O[mt][0];
          ow[(q0 + 1) * kHeadDim + 16 * mt + g] = st.O[mt][1];
          ow[q0 * kHeadDim + 16 * mt + g + 8] = st.O[mt][2];
          ow[(q0 + 1) * kHeadDim + 16 * mt + g + 8] = st.O[mt][3];
        }
      }
      __syncthreads();
      for (int q = 4 * pass; q < min(G, 4 * pass + 4); ++q) {
        float M = kNegInf;
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, merge_m[w * kMaxGroup + q]);
        float l = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) {
          const float mw = merge_m[w * kMaxGroup + q];
          const float al = mw == kNegInf ? 0.f : exp2f(mw - M);
          l += al * merge_l[w * kMaxGroup + q];
          o += al * merge_o[(w * 4 + (q - 4 * pass)) * kHeadDim + tid];
        }
        rec_o[(size_t(k) * G + q) * kHeadDim + tid] = o;
        if (tid == 0) {
          rec_m[size_t(k) * G + q] = M;
          rec_l[size_t(k) * G + q] = l;
        }
      }
    }
  }
}

template <int KB, int VB, bool ASYM, bool LOQ>
struct SuffixKernel {
  using T = SufFmt<KB, VB, ASYM>;
  static int smem_bytes(int B) { return suf_smem(kConsumerWarps * T::kRing, B, LOQ).total; }
  // CTAs of one wave on the current device.
  static int ctas(int B) {
    static std::mutex mu;
    static std::map<std::pair<int, int>, int> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lk(mu);
    const auto key = std::make_pair(dev, smem_bytes(B));
    auto it = done.find(key);
    if (it != done.end()) return it->second;
    int sms = 0, per = 0;
    const auto k = suffix_kernel<KB, VB, ASYM, LOQ>;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(4096)) != cudaSuccess ||
        cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k, kSufThreads, smem_bytes(B)) != cudaSuccess || per < 1)
      return 0;
    return done[key] = sms * per;
  }
  static cudaError_t launch(const SharedArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.sl.suf_ctas));
    cfg.blockDim = dim3(kSufThreads);
    cfg.dynamicSmemBytes = smem_bytes(a.d.B);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, suffix_kernel<KB, VB, ASYM, LOQ>, a);
  }
};

template <bool LOQ, class Fn>
auto suffix_by_format(const CacheView& c, Fn f) {
  const int kb = c.k_bits, vb = c.v_bits;
  const bool as = c.asym != 0;
  if (kb == 8 && vb == 8) return as ? f(SuffixKernel<8, 8, true, LOQ>{}) : f(SuffixKernel<8, 8, false, LOQ>{});
  if (kb == 4 && vb == 4) return as ? f(SuffixKernel<4, 4, true, LOQ>{}) : f(SuffixKernel<4, 4, false, LOQ>{});
  if (kb == 4 && vb == 8) return as ? f(SuffixKernel<4, 8, true, LOQ>{}) : f(SuffixKernel<4, 8, false, LOQ>{});
  if (kb == 8 && vb == 4) return as ? f(SuffixKernel<8, 4, true, LOQ>{}) : f(SuffixKernel<8, 4, false, LOQ>{});
  if (kb == 2 && vb == 2) return as ? f(SuffixKernel<2, 2, true, LOQ>{}) : f(SuffixKernel<2, 2, false, LOQ>{});
  return f(SuffixKernel<16, 16, false, false>{});
}

}  // namespace
}  // namespace kvq
