// Attention mass (kvq_attn_mass): the weight that every cached token received
// in a decode step, added to its running sum.
//
//   mass[b][h][i] = decay * mass[b][h][i] + sum_g exp(q_g . k_hat_i / sqrt(D) - lse_g)
//
// over the G query heads g of KV head h, with the log-sum-exp of each query that
// kvq_decode has written.  With the log-sum-exp known every token stands alone:
// no maximum, no merge, no atomics, one pass over the keys (the values are
// not read).  Bound: HBM, the key codes and scales plus 8 bytes of mass a token.
//
// Measured: 4 sequences of 131072 tokens, int4 keys, 64 query heads: 66 us, 319 MB at 4.8 TB/s (the copy rate
// would take 47); 32 of 1k-8k, int4: 26 us (13.6).  180 instructions a block, about 80 of them the exact conversion
// of 4-bit codes, keep the issue slots 58 % and the ALU 49 % busy: neither is full, but with 16 warps an SM the waits of
// one instruction on another are not covered (the query group and two blocks in flight are 128 registers; at 85 they
// spill and it takes 136 us).
//
// Work: the 16-token blocks of all (sequence, KV head) units, two a step, form one range cut
// evenly over all warps of one wave.  A warp keeps its unit's query
// group in registers as the B operand of m16n8k16 (tokens on M, queries on N) and streams blocks
// through its own ring of shared-memory stages with 16-byte asynchronous
// copies; the fragment-native block order gives each lane the bytes it copied
// itself.  (One block a step, the stages unrolled: 268 instructions a block, 99 us.)  Scores as in the decode kernel: exact codes in fp16, the key
// scale after the dot product.  The query is exact in fp16 (bf16 has 8
// significant bits) unless a per-channel key factor is folded in: then it is
// carried as an fp16 high and low part, because a weight's relative error is
// the score's absolute one.
#include "kvq_decode_impl.cuh"

namespace kvq {
namespace {

constexpr int kMassWarps = 8;
constexpr int kMassThreads = kMassWarps * 32;

template <int KB>
struct MassFmt {
  static constexpr bool kBf16 = KB == 16, kGroup = KB == 2;
  // Blocks of a step, copied and worked on together: the two blocks' chains of loads, products, exponentials
  // and shuffles overlap, and the sums of 32 tokens end up one in each lane.
  static constexpr int kNB = kBf16 ? 1 : 2;
  static constexpr int kRaw = block_bytes(KB);  // key codes of one block
  static constexpr int kChunks = kRaw / 512;
  static constexpr int kSide = 192;             // scales, zero points, mass: 16 floats each
  static constexpr int kOffSide = kNB * kRaw, kOffKo = 64, kOffMass = 128;
  static constexpr int kStageBytes = kOffSide + kNB * kSide;
  static constexpr int kStages = KB == 16 ? 2 : (KB == 8 ? 3 : 4);
  static constexpr int kRingBytes = kStages * kStageBytes * kMassWarps;
};

// S^T of one block as in score_block, from a stage in shared memory; the low
// query parts stay in registers here.
template <int KB, bool LOQ>
__device__ __forceinline__ void mass_scores(const uint8_t* kb, const uint32_t (&qf)[16], const uint32_t (&ql)[LOQ ? 16 : 1],
                                            float (&acc)[4], int lane, uint32_t km) {
  const uint4* p = reinterpret_cast<const uint4*>(kb) + lane;
  float acc2[4] = {0.f, 0.f, 0.f, 0.f};
  acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
  auto mma = [&](int kk, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
    float(&d)[4] = (kk & 1) ? acc2 : acc;
    if constexpr (KB == 16) {
      mma_bf16(d, a0, a1, a2, a3, qf[2 * kk], qf[2 * kk + 1]);
    } else {
      mma_f16(d, a0, a1, a2, a3, qf[2 * kk], qf[2 * kk + 1]);
      if constexpr (LOQ) mma_f16(d, a0, a1, a2, a3, ql[2 * kk], ql[2 * kk + 1]);
    }
  };
  if constexpr (KB == 8) {
    const uint4 r0a = p[0], r0b = p[32], r1a = p[64], r1b = p[96];
    const uint32_t g0[8] = {r0a.x, r0a.y, r0a.z, r0a.w, r0b.x, r0b.y, r0b.z, r0b.w};
    const uint32_t g8[8] = {r1a.x, r1a.y, r1a.z, r1a.w, r1b.x, r1b.y, r1b.z, r1b.w};
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      uint32_t a0, a1, a2, a3;
      s8x4_to_f16(g0[kk], a0, a2);
      s8x4_to_f16(g8[kk], a1, a3);
      mma(kk, a0, a1, a2, a3);
    }
  } else if constexpr (KB == 4) {
    const uint4 r0 = p[0], r1 = p[32];
    const uint32_t g0[4] = {r0.x, r0.y, r0.z, r0.w}, g8[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int wi = 0; wi < 4; ++wi) {
      uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
      s4x8_to_f16(g0[wi], km, x0, x1, x2, x3);
      s4x8_to_f16(g8[wi], km, y0, y1, y2, y3);
      mma(2 * wi, x0, y0, x1, y1);
      mma(2 * wi + 1, x2, y2, x3, y3);
    }
  } else if constexpr (KB == 2) {
    const uint4 r = p[0];
    const uint32_t wd[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int wi = 0; wi < 4; ++wi) {
      uint32_t o[8];
      s2x16_to_f16(wd[wi], km, o);
      mma(2 * wi, o[0], o[1], o[2], o[3]);
      mma(2 * wi + 1, o[4], o[5], o[6], o[7]);
    }
  } else {
    uint4 c[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) c[h] = p[h * 32];
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const uint4 lo = c[kk >> 1], hi = c[4 + (kk >> 1)];
      mma(kk, (kk & 1) ? lo.z : lo.x, (kk & 1) ? hi.z : hi.x, (kk & 1) ? lo.w : lo.y, (kk & 1) ? hi.w : hi.y);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] += acc2[i];
}

// The query group of unit (b, h) as this lane's B operand registers (query g,
// dims 32t..32t+31), and the score scale, the query sum (zero points) and the log-sum-exp
// (base 2) of queries 2t and 2t + 1.
template <int KB, bool ASYM, bool LOQ>
struct MassQuery {
  uint32_t qf[16];
  uint32_t ql[LOQ ? 16 : 1];
  float qs[2], qz[2], ls[2];

  __device__ __forceinline__ void load(const MassArgs& a, int b, int h, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const bool act = g < a.G;
    float x[32];
    const size_t row = size_t(b) * a.Hq + h * a.G + (act ? g : 0);
    const uint4* src = reinterpret_cast<const uint4*>(a.q + row * kHeadDim + 32 * t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = src[i];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = act ? __uint_as_float(w[j] << 16) : 0.f;
        x[8 * i + 2 * j + 1] = act ? __uint_as_float(w[j] & 0xFFFF0000u) : 0.f;
      }
    }
    if (KB != 16 && a.c.factor) {
      const float4* f = reinterpret_cast<const float4*>(a.c.factor + h * kHeadDim + 32 * t);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 c = f[i];
        x[4 * i] *= c.x;
        x[4 * i + 1] *= c.y;
        x[4 * i + 2] *= c.z;
        x[4 * i + 3] *= c.w;
      }
    }
    float scale = kLog2e * kInvSqrtD, z = 0.f;
    if (KB != 16 || a.c.q_bits == 8) {
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) am = fmaxf(am, fabsf(x[i]));
      am = fmaxf(am, __shfl_xor_sync(kFull, am, 1));
      am = fmaxf(am, __shfl_xor_sync(kFull, am, 2));
      if (a.c.q_bits == 8) {  // int8 query rows, as the decode kernel quantizes them
        float s = 1.f;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float y[4] = {x[i], x[i + 1], x[i + 2], x[i + 3]};
          float c[4];
          s = quantize_int8_row(y, am, c);
          x[i] = c[0];
          x[i + 1] = c[1];
          x[i + 2] = c[2];
          x[i + 3] = c[3];
        }
        scale *= s;
      } else if (am > 0.f) {
        int ex;
        frexpf(am, &ex);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = ldexpf(x[i], 15 - ex);
        scale = ldexpf(scale, ex - 15);
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (KB == 16) {
        qf[i] = pack_bf162(x[2 * i], x[2 * i + 1]);
      } else {
        qf[i] = pack_half2(x[2 * i], x[2 * i + 1]);
        const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&qf[i]));
        z += hi.x + hi.y;
        if constexpr (LOQ) {
          ql[i] = pack_half2(x[2 * i] - hi.x, x[2 * i + 1] - hi.y);
          const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&ql[i]));
          z += lo.x + lo.y;
        }
      }
    }
    float l = act ? a.lse[row] : 0.f;
    // no query in this column, or a query that attended to nothing: no weight
    l = act && l != kNegInf ? l * kLog2e : -kNegInf;
    if constexpr (ASYM) {
      z += __shfl_xor_sync(kFull, z, 1);
      z += __shfl_xor_sync(kFull, z, 2);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      qs[j] = __shfl_sync(kFull, scale, 4 * (2 * t + j));
      ls[j] = __shfl_sync(kFull, l, 4 * (2 * t + j));
      qz[j] = ASYM ? __shfl_sync(kFull, z, 4 * (2 * t + j)) : 0.f;
    }
  }
};

// The length of sequence b, clamped to the table's (its last tokens are in the ring, whatever a row of sums holds);
// `bad` reports one beyond the table or the row.
__device__ __forceinline__ int mass_len(const MassArgs& a, int b, bool& bad) {
  const int L = a.seq_lens[b], room = table_tokens(a.mbps, a.c.window);
  bad = bad || L < 0 || L > min(room, a.stride);
  return min(max(L, 0), room);
}

// Where a warp's copying or computing side is: step j of n, of unit (b, h).
struct MassPlace {
  int b, h, j, n;
  // to the next step of a range that ends after `left` more; whether the unit changed
  __device__ __forceinline__ bool advance(const int* pre, int H, bool more) {
    if (++j < n) return false;
    j = 0;
    if (++h == H) {
      h = 0;
      if (more) {
        do { ++b; } while (pre[b + 1] == pre[b]);
        n = pre[b + 1] - pre[b];
      }
    }
    return true;
  }
};

// RING: the blocks are those of the bf16 window (KB = 16).
template <int KB, bool ASYM, bool LOQ, bool RING>
__global__ void __launch_bounds__(kMassThreads) mass_kernel(const MassArgs a) {
  using F = MassFmt<KB>;
  constexpr int NB = F::kNB;
  extern __shared__ __align__(128) uint8_t smem[];
  int* pre = reinterpret_cast<int*>(smem + F::kRingBytes);  // [B + 1] steps of one head before sequence b
  int* lens = pre + a.B + 1;                                // [B]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int B = a.B, H = a.c.H, W = a.c.window;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  bool bad = false;
  for (int b = tid; b < B; b += kMassThreads) {
    const int L = mass_len(a, b, bad);
    const int n = RING ? min(L, W) : min(max(L - W, 0), a.stride);
    lens[b] = L;
    pre[b + 1] = (n + kBlock * NB - 1) / (kBlock * NB);
  }
  if (bad && blockIdx.x == 0) flag(a.err, KVQ_DEVERR_SEQ_LEN);
  if (tid == 0) pre[0] = 0;
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base < B; base += 32) {
      const int i = base + lane;
      int v = i < B ? pre[i + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += n;
      }
      if (i < B) pre[i + 1] = v + carry;
      carry += __shfl_sync(kFull, v, 31);
    }
  }
  __syncthreads();
  const long long T = (long long)H * pre[B];
  const long long NW = (long long)gridDim.x * kMassWarps, w = (long long)blockIdx.x * kMassWarps + warp;
  const long long x0 = w * T / NW;
  const int steps = int((w + 1) * T / NW - x0);
  if (steps <= 0) return;

  // unit of step x0: the largest b with H * pre[b] <= x0 that has blocks
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)H * pre[mid] <= x0) lo = mid;
    else hi = mid - 1;
  }
  while (pre[lo + 1] == pre[lo]) ++lo;
  const int first_n = pre[lo + 1] - pre[lo];
  const int first_x = int(x0 - (long long)H * pre[lo]);
  MassPlace in{lo, first_x / first_n, first_x % first_n, first_n}, at = in;

  // ---- the copying side
  uint8_t* const ring = smem + warp * (F::kStages * F::kStageBytes);
  const uint8_t* codes = nullptr;  // this lane's first piece of block 0 of the head, of its window
  const float* side = nullptr;     // this lane's piece of the head's block 0 record, or of the unit's mass
  const int* table = nullptr;
  int blocks = 0;
  // lanes 12 i + r: pieces of block i's scales and zero points (r < 8) and mass
  const int side_i = lane >= 12, side_r = lane - 12 * side_i;
  const bool side_mass = side_r >= 8;
  const bool side_on = !RING && lane < 12 * NB &&
                       (side_mass || (!F::kBf16 && !a.c.k_chan && side_r < (F::kGroup ? 1 : (ASYM ? 8 : 4))));
  const int side_step = side_mass ? kBlock : a.c.meta_floats;
  int ids = -1, ids_next = -1, ids_base = 0;  // 32 table entries, and the 32 behind them on their way
  auto entry = [&](int i) { return i + lane < blocks ? table[i + lane] : -1; };
  auto check = [&](int i) {
    if (i + lane < blocks && (ids < 0 || ids >= a.c.num_blocks)) {
      flag(a.err, KVQ_DEVERR_BLOCK_ID);
      ids = -1;
    }
  };
  auto enter = [&]() {
    const size_t unit = size_t(in.b) * H + in.h;
    if constexpr (RING) {
      codes = a.c.k_win + unit * (W / kBlock) * F::kRaw + lane * 16;
    } else {
      const size_t hb = size_t(in.h) * a.c.num_blocks;
      codes = a.c.k_codes + hb * F::kRaw + lane * 16;
      side = side_mass ? a.mass + unit * a.stride + (side_r - 8) * 4 : a.c.meta + hb * a.c.meta_floats + side_r * 4;
      table = a.table + size_t(in.b) * a.mbps;
      blocks = (lens[in.b] - W + kBlock - 1) / kBlock;
      ids_base = in.j * NB;
      ids = entry(ids_base);
      ids_next = entry(ids_base + 32);
      check(ids_base);
    }
  };
  enter();
  uint32_t valid = 0u;  // blocks of the ring's stages that are to be read (a bad table entry is not)
  int s_in = 0, left = steps;
  auto fetch = [&]() {
    if (left > 0) {
      uint8_t* st = ring + s_in * F::kStageBytes;
      const int j = in.j * NB;
      if constexpr (!RING) {
        if (j - ids_base == 32) {
          ids_base = j;
          ids = ids_next;
          ids_next = entry(j + 32);
          check(j);
        }
      }
      uint32_t ok = 0u;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int phys = RING ? j : __shfl_sync(kFull, ids, j - ids_base + i);
        if (phys >= 0) {
          ok |= 1u << i;
          const uint8_t* src = codes + size_t(phys) * F::kRaw;
#pragma unroll
          for (int c = 0; c < F::kChunks; ++c) cp_async16(st + i * F::kRaw + lane * 16 + c * 512, src + c * 512);
        }
      }
      valid = (valid & ~(((1u << NB) - 1u) << (s_in * NB))) | (ok << (s_in * NB));
      if constexpr (!RING) {
        const int phys = __shfl_sync(kFull, ids, j - ids_base + (NB > 1 ? side_i : 0));
        const int blk = side_mass ? j + side_i : phys;
        // the row may end inside its last block
        if (side_on && phys >= 0 && (!side_mass || blk * kBlock + (side_r - 8) * 4 < a.stride))
          cp_async16(st + F::kOffSide + side_i * F::kSide + side_r * 16, side + (long long)blk * side_step);
      }
      --left;
      if (in.advance(pre, H, left > 0) && left > 0) enter();
      if (++s_in == F::kStages) s_in = 0;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < F::kStages - 1; ++i) fetch();

  // ---- the computing side
  const uint32_t km = magic_f16x2(B);
  MassQuery<KB, ASYM, LOQ> mq;
  mq.load(a, at.b, at.h, lane);
  float* row = a.mass + (size_t(at.b) * H + at.h) * a.stride;
  auto length = [&](int b) { return RING ? lens[b] : min(lens[b] - W, a.stride); };  // of the unit; its stored tokens in the row
  int L = length(at.b), s = 0;
  // not unrolled over the stages: the code of one step has to stay in the instruction cache
#pragma unroll 1
  for (int x = steps; x > 0; --x) {
    fetch();  // the step after the ring's others goes into the stage freed last
    cp_async_wait<F::kStages - 1>();
    __syncwarp();
    const uint8_t* st = ring + s * F::kStageBytes;
    float wt[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float acc[4];
      mass_scores<KB, LOQ>(st + n * F::kRaw, mq.qf, mq.ql, acc, lane, km);
      const float* ks = reinterpret_cast<const float*>(st + F::kOffSide + n * F::kSide);
      float sk[2] = {1.f, 1.f}, mk[2] = {0.f, 0.f};
      if (!F::kBf16 && !a.c.k_chan) {
        sk[0] = ks[F::kGroup ? 0 : g];
        sk[1] = ks[F::kGroup ? 0 : g + 8];
        if (ASYM) {
          constexpr float kKC = KB == 8 ? 128.f : (KB == 4 ? 8.f : 2.f);
          const float* ko = F::kGroup ? ks + 1 : ks + F::kOffKo / 4;
          mk[0] = fmaf(kKC, sk[0], ko[F::kGroup ? 0 : g]);
          mk[1] = fmaf(kKC, sk[1], ko[F::kGroup ? 0 : g + 8]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // token g, g + 8
        wt[n][i] = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // query 2t, 2t + 1
          const float v = ASYM ? fmaf(acc[2 * i + c], sk[i], mk[i] * mq.qz[c]) : acc[2 * i + c] * sk[i];
          wt[n][i] += ex2(fmaf(v, mq.qs[c], -mq.ls[c]));
        }
      }
    }
    // sums over the four lanes of a token: lane t ends with token g + 8 (t & 1) of block t >> 1
    float add[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n)
      add[n] = ((t & 1) ? wt[n][1] : wt[n][0]) + __shfl_xor_sync(kFull, (t & 1) ? wt[n][0] : wt[n][1], 1);
    float sum;
    if constexpr (NB == 2) {
      sum = ((t & 2) ? add[1] : add[0]) + __shfl_xor_sync(kFull, (t & 2) ? add[0] : add[1], 2);
    } else {
      sum = add[0] + __shfl_xor_sync(kFull, add[0], 2);
    }
    const int n = NB == 2 ? t >> 1 : 0, tok = g + 8 * (t & 1), slot = (at.j * NB + n) * kBlock + tok;
    if ((valid >> (s * NB + n) & 1u) && (NB == 2 || t < 2)) {
      if constexpr (RING) {  // ring tokens' slots are not in order of their positions
        const int first = L - min(L, W), p = first + ((slot - first) % W + W) % W;
        if (p < min(L, a.stride)) row[p] = fmaf(a.decay, row[p], sum);
      } else {
        const float old = reinterpret_cast<const float*>(st + F::kOffSide + n * F::kSide + F::kOffMass)[tok];
        if (slot < L) row[slot] = fmaf(a.decay, old, sum);
      }
    }
    __syncwarp();  // every lane has read the stage before it is filled again
    if (++s == F::kStages) s = 0;
    if (at.advance(pre, H, x > 1) && x > 1) {
      L = length(at.b);
      row = a.mass + (size_t(at.b) * H + at.h) * a.stride;
      mq.load(a, at.b, at.h, lane);
    }
  }
}

template <int KB, bool ASYM, bool LOQ, bool RING>
cudaError_t launch_one(const MassArgs& a, cudaStream_t s) {
  using F = MassFmt<KB>;
  const int smem = F::kRingBytes + (2 * a.B + 1) * 4;
  static std::mutex mu;
  static std::map<std::pair<int, int>, int> grids;  // CTAs of one wave, by device and shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int grid = 0;
  {
    std::lock_guard<std::mutex> lk(mu);
    auto it = grids.find({dev, smem});
    if (it == grids.end()) {
      int sms = 0, per = 0;
      if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
      e = cudaFuncSetAttribute(mass_kernel<KB, ASYM, LOQ, RING>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               F::kRingBytes + (2 * kMaxBatch + 1) * 4);
      if (e != cudaSuccess) return e;
      e = cudaFuncSetAttribute(mass_kernel<KB, ASYM, LOQ, RING>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
      if (e != cudaSuccess) return e;
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, mass_kernel<KB, ASYM, LOQ, RING>, kMassThreads, smem);
      if (e != cudaSuccess) return e;
      it = grids.emplace(std::make_pair(dev, smem), sms * (per < 1 ? 1 : per)).first;
    }
    grid = it->second;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMassThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mass_kernel<KB, ASYM, LOQ, RING>, a);
}

template <int KB>
cudaError_t launch_codes(const MassArgs& a, cudaStream_t s) {
  const bool lo = a.c.factor && a.c.q_bits != 8;  // int8 query rows are exact in fp16
  if (a.c.asym) return lo ? launch_one<KB, true, true, false>(a, s) : launch_one<KB, true, false, false>(a, s);
  return lo ? launch_one<KB, false, true, false>(a, s) : launch_one<KB, false, false, false>(a, s);
}

}  // namespace

cudaError_t launch_mass(const MassArgs& a, cudaStream_t s) {
  if (a.c.window > 0) {
    const cudaError_t e = launch_one<16, false, false, true>(a, s);
    if (e != cudaSuccess) return e;
  }
  switch (a.c.k_bits) {
    case 2: return launch_codes<2>(a, s);
    case 4: return launch_codes<4>(a, s);
    case 8: return launch_codes<8>(a, s);
    default: return launch_one<16, false, false, false>(a, s);
  }
}

}  // namespace kvq
