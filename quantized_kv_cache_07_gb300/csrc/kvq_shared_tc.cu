// The shared prefix of kvq_decode_shared on tcgen05, for groups of many query vectors.
//
// A CTA takes 128 query vectors of one group and KV head and streams its share
// of the prefix 64 tokens (4 blocks) at a time:
//   S (128 x 64, tensor memory) = Q (fp16, shared memory) . K^T (codes converted to fp16, shared memory)
//   P = exp2(S * s_k * scale - m), one thread per query vector, fp16 weights P * s_v back to tensor memory
//   O (128 x 128, tensor memory) += P . V (codes converted to fp16, shared memory)
// Each block is converted once for 128 vectors; on mma.sync every 16 vectors
// convert it again, and that conversion is what bounds the 16-vector tiles.
//
// Roles: warps 0-3 softmax (thread v = vector v = tensor-memory lane v), warps
// 4-7 conversion (warp w = block w of the 64 tokens, the next tile's codes already in
// registers).  Threads of warps 0 and 1 issue the products between their own steps (a ninth
// warp would cost every thread 32 of its 128 registers).  K, V and S are double-buffered; P overwrites its S.  256 columns of tensor memory
// and about 105 KB of shared memory: two CTAs share an SM and fill each other's waits.
//
// Orders inside a tile.  The tokens and dims of a block are permuted so that a lane's codes
// (fragment-native order, include/kvq.h) go to shared memory as 16-byte (K) and
// 8-byte (V) stores without bank conflicts:
//   token i of block b:  column 8 b + 32 (t >> 1) + 4 (t & 1) + j,  t = (i & 7) >> 1, j = 2 (i & 1) + (i >> 3)
//   dim 32 t + 8 i + e:  half i >> 1, 16-byte chunk (t & 1) + 4 (t >> 1) + 2 (i & 1), element e
// (the same dim order for Q and K; the same token order for the columns of S and the k-index of P . V).
//
// Precision as in the decode kernel: exact codes, the query exact in fp16 (or
// int8 codes), scales in fp32, fp16 weights kept in range by the sigma offset
// (kvq_decode_impl.cuh), fp32 sums of the unrounded weights.
#include "kvq_shared.cuh"
#include "kvq_tcgen05.cuh"
#include "kvq_tiles.cuh"

namespace kvq {
namespace {

constexpr int kQ = 128;            // query vectors of a unit
constexpr int kTok = 64;           // tokens of a tile
constexpr int kTcThreads = 256;
constexpr int kTmemCols = 256;     // O: 0..127, S buffers: 128.., 192..
constexpr int kScaleRing = 4;      // a tile's scales are written two tiles ahead of its predecessor's last reader

struct TcSmem {
  alignas(1024) uint8_t q[2][kQ * 128];      // two halves of 64 dims
  alignas(1024) uint8_t k[2][2][kTok * 128];  // [buffer][half]
  alignas(1024) uint8_t v[2][kHeadDim * 128];
  float sk[kScaleRing][kTok], sv[kScaleRing][kTok], mk[kScaleRing][kTok], mv[kScaleRing][kTok];
  float svmax[kScaleRing][4];
  float qs[kQ], qz[kQ];
  int qlen[kQ];
  uint64_t k_full[4];  // by tile & 3: a softmax warp may look after the conversion has run two tiles ahead
  uint64_t v_full[2], qk_done[2], p_full[2], pv_done[2];
  uint32_t tmem;
  int dead;
  int maxlen, minlen;
  SharedGeo geo;
};

// Two float32 operations in one instruction, in place on (x, y).
__device__ __forceinline__ void fma2(uint32_t& x, uint32_t& y, float ax, float ay, float bx, float by) {
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n mov.b64 c, {%4, %5};\n"
      " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}"
      : "+r"(x), "+r"(y)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by));
}
__device__ __forceinline__ void mul2(uint32_t& x, uint32_t& y, float ax, float ay) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n"
      " mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "+r"(x), "+r"(y)
      : "f"(ax), "f"(ay));
}
__device__ __forceinline__ void add2(uint32_t& x, uint32_t& y, uint32_t ax, uint32_t ay) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n"
      " add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "+r"(x), "+r"(y)
      : "r"(ax), "r"(ay));
}

// Column of token i of block b in a tile.
__host__ __device__ constexpr int tile_col(int b, int i) {
  return 8 * b + 32 * ((i & 7) >> 2) + 4 * (((i & 7) >> 1) & 1) + 2 * (i & 1) + (i >> 3);
}
// Token (within the tile) of column n.
__host__ __device__ constexpr int tile_token(int n) {
  return 16 * ((n >> 3) & 3) + 2 * (2 * (n >> 5) + ((n >> 2) & 1)) + ((n & 3) >> 1) + 8 * (n & 1);
}
static_assert(tile_token(40) == tile_token(8) + 4, "the upper 32 columns hold the same blocks' tokens, four on");
static_assert(tile_token(tile_col(3, 13)) == 61 && tile_token(tile_col(0, 6)) == 6 && tile_token(tile_col(2, 9)) == 41,
              "column order");

__device__ __forceinline__ uint32_t dim_chunk(int t, int i) { return (t & 1) | ((t >> 1) << 2) | ((i & 1) << 1); }

// One lane's raw codes of a block: 16-byte pieces of the fragment-native order.
template <int BITS>
struct Raw {
  static constexpr int kPieces = BITS / 2;
  uint4 p[kPieces];
  __device__ __forceinline__ void load(const uint8_t* blk, int lane) {
#pragma unroll
    for (int c = 0; c < kPieces; ++c) p[c] = __ldcg(reinterpret_cast<const uint4*>(blk) + c * 32 + lane);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int c = 0; c < kPieces; ++c) p[c] = make_uint4(0u, 0u, 0u, 0u);
  }
};

// Keys of block w to the K tile (lane (g, t): tokens g and g + 8, dims 32t..32t+31).
template <int KB>
__device__ __forceinline__ void put_keys(const Raw<KB>& raw, uint8_t* const half0, uint8_t* const half1, int w, int lane,
                                         uint32_t km, uint32_t c64) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    const int row = tile_col(w, g + 8 * hi);
    auto put = [&](int i, uint4 v) {
      uint8_t* base = (i >> 1) ? half1 : half0;
      *reinterpret_cast<uint4*>(base + row * 128 + ((dim_chunk(t, i) ^ (row & 7)) * 16)) = v;
    };
    if constexpr (KB == 8) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 r = raw.p[2 * hi + c];
        uint4 o;
        s8x4_to_f16_r(r.x, c64, o.x, o.y);
        s8x4_to_f16_r(r.y, c64, o.z, o.w);
        put(2 * c, o);
        s8x4_to_f16_r(r.z, c64, o.x, o.y);
        s8x4_to_f16_r(r.w, c64, o.z, o.w);
        put(2 * c + 1, o);
      }
    } else if constexpr (KB == 4) {
      const uint4 r = raw.p[hi];
      const uint32_t wd[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 o;
        s4x8_to_f16(wd[i], km, o.x, o.y, o.z, o.w);
        put(i, o);
      }
    } else {
      const uint4 r = raw.p[0];
      const uint32_t wd[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[8];
        s2x16_to_f16(wd[i], km, o);
        put(i, make_uint4(o[hi], o[hi + 2], o[4 + hi], o[6 + hi]));
      }
    }
  }
}

// Values of block w to the V tile (rows: dims, 64 tokens each; lane (g, t): dims 16 mt + g (+ 8), four tokens).
template <int VB>
__device__ __forceinline__ void put_values(const Raw<VB>& raw, uint8_t* const tile, int w, int lane, uint32_t km,
                                           uint32_t c64) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t at = (((w + 4 * (t >> 1)) ^ g) * 16) + 8 * (t & 1);
  auto put = [&](int d, uint32_t lo, uint32_t hi) { *reinterpret_cast<uint2*>(tile + d * 128 + at) = make_uint2(lo, hi); };
  if constexpr (VB == 8) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t wd[4] = {raw.p[c].x, raw.p[c].y, raw.p[c].z, raw.p[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        s8x4_to_f16_r(wd[i], c64, lo, hi);
        put(16 * (2 * c + (i >> 1)) + 8 * (i & 1) + g, lo, hi);
      }
    }
  } else if constexpr (VB == 4) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t wd[4] = {raw.p[c].x, raw.p[c].y, raw.p[c].z, raw.p[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a, b, d, e;
        s4x8_to_f16(wd[i], km, a, b, d, e);
        put(16 * (4 * c + i) + g, a, b);
        put(16 * (4 * c + i) + 8 + g, d, e);
      }
    }
  } else {
    const uint32_t wd[4] = {raw.p[0].x, raw.p[0].y, raw.p[0].z, raw.p[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t o[8];
      s2x16_to_f16(wd[i], km, o);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) put(16 * (2 * i + h) + 8 * hi + g, o[4 * h + hi], o[4 * h + hi + 2]);
    }
  }
}

// Query vector v (this lane's four bf16 values in raw) into the swizzled Q tile by one warp; returns its score scale.
template <bool ASYM>
__device__ __forceinline__ float put_query(const DecodeArgs& a, uint2 raw, float4 c, int v, TcSmem* sm, int lane) {
  float x[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u), __uint_as_float(raw.y << 16),
                __uint_as_float(raw.y & 0xFFFF0000u)};
  if (a.c.factor) {
    x[0] *= c.x;
    x[1] *= c.y;
    x[2] *= c.z;
    x[3] *= c.w;
  }
  // non-negative floats order as their bits: one warp reduction
  const float am = __uint_as_float(__reduce_max_sync(
      kFull, __float_as_uint(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))))));
  float scale = kLog2e * kInvSqrtD;
  if (a.c.q_bits == 8) {
    float q[4];
    scale *= quantize_int8_row(x, am, q);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = q[j];
  } else {
    // exact powers of two: am * 2^(14 - e) in [2^14, 2^15); below 2^-112 the scores are zero to any precision
    const uint32_t e = max(__float_as_uint(am) >> 23, 15u);
    const float f = __uint_as_float((268u - e) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] *= f;
    scale *= __uint_as_float((e - 14u) << 23);
  }
  const uint2 y = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
  if constexpr (ASYM) {  // the vector's sum as the product sees it
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&y.x));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&y.y));
    float z = (f0.x + f0.y) + (f1.x + f1.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
    if (lane == 0) sm->qz[v] = z;
  }
  const int t = lane >> 3, i = (lane & 7) >> 1;
  *reinterpret_cast<uint2*>(sm->q[i >> 1] + v * 128 + ((dim_chunk(t, i) ^ (v & 7)) * 16) + 8 * (lane & 1)) = y;
  return fmaxf(scale, 1.17549435e-38f);  // positive, so that a masked score stays -inf
}

template <int KB, int VB, bool ASYM>
__global__ void __launch_bounds__(kTcThreads, 2) shared_tc_kernel(const SharedArgs sa) {
  using F = Fmt<KB, VB, ASYM>;
  constexpr int kStep = kTok / kBlock;
  constexpr float kKC = KB == 8 ? 128.f : (KB == 4 ? 8.f : 2.f), kVC = VB == 8 ? 128.f : (VB == 4 ? 8.f : 2.f);
  const DecodeArgs& a = sa.d;
  extern __shared__ uint8_t raw_smem[];
  TcSmem* sm = reinterpret_cast<TcSmem*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  const int G = a.G, H = a.c.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(&sm->k_full[i], 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->v_full[i], 128);
      mbar_init(&sm->qk_done[i], 1);
      mbar_init(&sm->p_full[i], 128);
      mbar_init(&sm->pv_done[i], 1);
    }
    sm->dead = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  shared_geometry(&sm->geo, a, kQ, kStep, tid, kTcThreads, false);  // errors are reported by the suffix decode
  const SharedGeo* geo = &sm->geo;
  const int Pe = shared_ctas(geo, sa.sl.ctas), ci = blockIdx.x;
  if (ci >= Pe) return;
  const long long x0 = (long long)ci * geo->T / Pe, x1 = (long long)(ci + 1) * geo->T / Pe;
  if (x0 >= x1) return;
  if (warp == 4) tmem_alloc(&sm->tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem;
  const uint32_t km = magic_f16x2(a.B);
  const uint32_t c64 = 0x64646464u | (uint32_t(a.B) >> 16);  // a.B <= 4096: the constant itself

  int it = 0;  // tiles of the CTA so far: buffer it & 1, phase (it >> 1) & 1
  auto wait = [&](uint64_t* bars, int i) { return mbar_wait(&bars[i & 1], uint32_t(i >> 1) & 1u); };
  auto wait_k = [&](int i) { return mbar_wait(&sm->k_full[i & 3], uint32_t(i >> 2) & 1u); };
  auto give_up = [&]() {
    flag(a.err, KVQ_DEVERR_TIMEOUT);
    sm->dead = 1;
  };
  for (long long x = x0; x < x1;) {
    const SharedUnit un = unit_at(geo, a.num_groups, H, kStep, x);
    const int nt = int(min(x1, un.start + un.steps) - x);  // tiles of this segment
    const int t0 = int(x - un.start);                      // the first one's number in the unit
    x += nt;
    const int nblk = geo->g.blocks[un.group], first = geo->g.start[un.group];
    const int rows = geo->g.start[un.group + 1] - first;
    if (tid == 0) {
      sm->maxlen = 0;
      sm->minlen = 0x7fffffff;
    }
    __syncthreads();
    {
      // all of this warp's 16 vectors are loaded before the first is converted: one memory latency, not 16
      constexpr int kPer = kQ / (kTcThreads / 32);
      const uint16_t* q0 = a.q + (size_t(first) * a.Hq + un.h * G) * kHeadDim + 4 * lane;
      uint2 raw[kPer];
      int mylen = 0;  // lane i < 16: vector i's prefix length
      float4 c = make_float4(1.f, 1.f, 1.f, 1.f);
      if (a.c.factor) c = *reinterpret_cast<const float4*>(a.c.factor + un.h * kHeadDim + 4 * lane);
      const int gv0 = un.tile * kQ + warp * kPer;
      {
        const int rr = (gv0 + (lane & (kPer - 1))) / G;
        if (rr < rows) mylen = prefix_len(a, first + rr, nblk);
        if (lane < kPer) {
          sm->qlen[warp * kPer + lane] = mylen;
          atomicMax(&sm->maxlen, mylen);
          if (rr < rows) atomicMin(&sm->minlen, mylen);
        }
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int rr = (gv0 + i) / G, hj = (gv0 + i) % G;
        raw[i] = make_uint2(0u, 0u);
        if (rr < rows) raw[i] = *reinterpret_cast<const uint2*>(q0 + (size_t(rr) * a.Hq + hj) * kHeadDim);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float qs = put_query<ASYM>(a, raw[i], c, warp * kPer + i, sm, lane);
        if (lane == 0) sm->qs[warp * kPer + i] = qs;
      }
    }
    fence_async_smem();
    __syncthreads();

    if (warp >= 4) {
      // -------------------------------------------------------------- conversion
      const int w = warp - 4;
      const int* table = a.table + size_t(first) * a.mbps;
      const int maxlen = sm->maxlen;
      int ids = -1, ids_next = -1;  // this warp's table entries of 32 tiles, and of the next 32
      auto load_ids = [&](int i) {
        const int blk = (t0 + i + lane) * kStep + w;
        int id = -1;
        if (i + lane < nt && blk < nblk) {
          id = table[blk];
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
          ids_next = load_ids(i + 32);
        }
        return i < nt ? __shfl_sync(kFull, ids, i & 31) : -1;
      };
      auto fetch_keys = [&](int phys) {
        ks = vs = ko = vo = 0.f;
        rk.clear();
        if (phys < 0) return;
        const size_t hb = size_t(un.h) * a.c.num_blocks + phys;
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
        if (phys >= 0) rv.load(a.c.v_codes + (size_t(un.h) * a.c.num_blocks + phys) * F::kVBB, lane);
      };
      bool ok = true;
      {
        const int phys = block_of(0);
        fetch_keys(phys);
        fetch_values(phys);
      }
#pragma unroll 1
      for (int i = 0; i < nt; ++i) {
        const int n = it + i, b = n & 1, sc = n & (kScaleRing - 1);
        if (n >= 2 && !__all_sync(kFull, wait(sm->qk_done, n - 2))) {
          ok = false;
          break;
        }
        put_keys<KB>(rk, sm->k[b][0], sm->k[b][1], w, lane, km, c64);
        // scales of slots behind the longest row are not data
        const bool data = ((t0 + i) * kStep + w) * kBlock + lane < maxlen;
        if (!data) vs = 0.f;
        if (lane < kBlock) {
          const int col = tile_col(w, lane);
          sm->sk[sc][col] = ks;
          sm->sv[sc][col] = vs;
          if constexpr (ASYM) {
            sm->mk[sc][col] = fmaf(kKC, ks, ko);
            sm->mv[sc][col] = data ? fmaf(kVC, vs, vo) : 0.f;
          }
        }
        // value scales are positive: they order as their bits
        const uint32_t vm = __reduce_max_sync(kFull, lane < kBlock ? __float_as_uint(vs) : 0u);
        if (lane == 0) sm->svmax[sc][w] = __uint_as_float(vm);
        fence_async_smem();
        mbar_arrive(&sm->k_full[n & 3]);
        const int phys = block_of(i + 1);
        fetch_keys(phys);
        if (n >= 2 && !__all_sync(kFull, wait(sm->pv_done, n - 2))) {
          ok = false;
          break;
        }
        put_values<VB>(rv, sm->v[b], w, lane, km, c64);
        fence_async_smem();
        mbar_arrive(&sm->v_full[b]);
        fetch_values(phys);
      }
      if (!ok) give_up();
    } else {
      // -------------------------------------------------------------- softmax
      const int v = tid;
      const uint32_t lanes = tmem + (uint32_t(warp * 32) << 16);
      const float qs = sm->qs[v], qz = ASYM ? sm->qz[v] : 0.f;
      const int len = sm->qlen[v], minlen = sm->minlen;
      float m = kNegInf, l = 0.f, z = 0.f, sg = float(kSigma0);
      float svlim = ldexpf(1.f, kWeightExp - int(kMaxSlack) - kSigma0);
      bool ok = true;
      // S of tile i (issued by warp 1), and P . V of tile i (issued by warp 0): one thread each.  S's buffer is
      // free once P . V of tile i - 2 has read its weights.
      auto issue_qk = [&](int i) {
        if (warp != 1 || i >= nt) return;
        if (lane == 0) {
          const int n = it + i, b = n & 1;
          if (wait_k(n) && (n < 2 || wait(sm->pv_done, n - 2))) {
            tc_fence_after();
            const uint64_t qd = tile_desc(smem_u32(sm->q[0])), kd = tile_desc(smem_u32(sm->k[b][0]));
#pragma unroll
            for (int k = 0; k < kHeadDim / 16; ++k)
              tc_mma_ss(tmem + 128 + 64 * b, qd + (k >> 2) * (sizeof(sm->q[0]) >> 4) + 2 * (k & 3),
                        kd + (k >> 2) * (sizeof(sm->k[0][0]) >> 4) + 2 * (k & 3), f16_idesc(kQ, kTok), k > 0);
            tc_commit(&sm->qk_done[b]);
          } else {
            ok = false;
          }
        }
        __syncwarp();
      };
      auto issue_pv = [&](int i) {
        if (warp != 0) return;
        if (lane == 0) {
          const int n = it + i, b = n & 1;
          if (wait(sm->p_full, n) && wait(sm->v_full, n)) {
            tc_fence_after();
            const uint64_t vd = tile_desc(smem_u32(sm->v[b]));
#pragma unroll
            for (int k = 0; k < kTok / 16; ++k)
              tc_mma_ts(tmem, tmem + 128 + 64 * b + 8 * k, vd + 2 * k, f16_idesc(kQ, kHeadDim), i > 0 || k > 0);
            tc_commit(&sm->pv_done[b]);
          } else {
            ok = false;
          }
        }
        __syncwarp();
      };
      issue_qk(0);
      issue_qk(1);
      // O *= f, this thread's row; the products before tile i have to be complete
      auto rescale = [&](int i, float f) {
        if (i == 0) return true;
        if (!__all_sync(kFull, wait(sm->pv_done, it + i - 1))) return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 32) {
          uint32_t o[32];
          tmem_ld32(lanes + c, o);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          tmem_st32(lanes + c, o);
        }
        tc_wait_st();
        return true;
      };
      for (int i = 0; i < nt; ++i) {
        const int n = it + i, b = n & 1, sc = n & (kScaleRing - 1);
        ok = __all_sync(kFull, ok && wait_k(n) && wait(sm->qk_done, n));  // the scales, the scores
        if (!ok) break;
        tc_fence_after();
        const int tok0 = (t0 + i) * kTok;
        const uint32_t st = lanes + 128 + 64 * b;
        // 32 columns of S times their key scales (the zero-point terms added), masked
        auto scores = [&](int half, uint32_t (&r)[32]) {
          tmem_ld32(st + half, r);
          tc_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 ks = *reinterpret_cast<const float4*>(&sm->sk[sc][half + c]);
            if constexpr (ASYM) {
              const float4 ko = *reinterpret_cast<const float4*>(&sm->mk[sc][half + c]);
              fma2(r[c], r[c + 1], ks.x, ks.y, ko.x * qz, ko.y * qz);
              fma2(r[c + 2], r[c + 3], ks.z, ks.w, ko.z * qz, ko.w * qz);
            } else {
              mul2(r[c], r[c + 1], ks.x, ks.y);
              mul2(r[c + 2], r[c + 3], ks.z, ks.w);
            }
          }
          if (tok0 + kTok > minlen) {  // a row of the unit ends inside this tile or before it
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (tok0 + tile_token(c) + half / 8 >= len) r[c] = __float_as_uint(kNegInf);
          }
        };
        float mx = kNegInf;
#pragma unroll 1
        for (int half = 0; half < kTok; half += 32) {
          uint32_t r[32];
          scores(half, r);
          float m2 = kNegInf;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            mx = fmaxf(mx, fmaxf(__uint_as_float(r[c]), __uint_as_float(r[c + 1])));
            m2 = fmaxf(m2, fmaxf(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])));
          }
          mx = fmaxf(mx, m2);
        }
        mx *= qs;
        const float4 sm4 = *reinterpret_cast<const float4*>(sm->svmax[sc]);
        const float svm = fmaxf(fmaxf(sm4.x, sm4.y), fmaxf(sm4.z, sm4.w));
        if (__any_sync(kFull, mx > m + kMaxSlack) || svm > svlim) {  // svm is the same in every thread
          float f = 1.f;
          if (__any_sync(kFull, mx > m + kMaxSlack)) {
            const float mn = fmaxf(m, mx);
            f = mn == kNegInf ? 1.f : ex2(m - mn);
            m = mn;
          }
          if (svm > svlim) {
            int e;
            frexpf(svm, &e);
            const int sn = min(int(sg), kWeightExp - int(kMaxSlack) - e);
            f *= ldexpf(1.f, sn - int(sg));
            sg = float(sn);
            svlim = ldexpf(1.f, kWeightExp - int(kMaxSlack) - sn);
          }
          l *= f;
          z *= f;
          ok = rescale(i, f);
          if (!ok) break;
        }
        if (i > 0) issue_qk(i + 1);  // by now P . V of tile i - 1 has most likely finished
        const float base = m == kNegInf ? 0.f : m - sg;
        uint32_t la[4] = {0u, 0u, 0u, 0u};  // four partial sums of the weights
#pragma unroll 1
        for (int half = 0; half < kTok; half += 32) {
          uint32_t r[32], p[16];
          scores(half, r);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 vs = *reinterpret_cast<const float4*>(&sm->sv[sc][half + c]);
            fma2(r[c], r[c + 1], qs, qs, -base, -base);
            fma2(r[c + 2], r[c + 3], qs, qs, -base, -base);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[c + j] = __float_as_uint(ex2(__uint_as_float(r[c + j])));
            add2(la[0], la[1], r[c], r[c + 1]);
            add2(la[2], la[3], r[c + 2], r[c + 3]);
            if constexpr (ASYM) {
              const float4 vo = *reinterpret_cast<const float4*>(&sm->mv[sc][half + c]);
              z = fmaf(__uint_as_float(r[c]), vo.x, fmaf(__uint_as_float(r[c + 1]), vo.y, z));
              z = fmaf(__uint_as_float(r[c + 2]), vo.z, fmaf(__uint_as_float(r[c + 3]), vo.w, z));
            }
            mul2(r[c], r[c + 1], vs.x, vs.y);
            mul2(r[c + 2], r[c + 3], vs.z, vs.w);
            p[c / 2] = pack_half2(__uint_as_float(r[c]), __uint_as_float(r[c + 1]));
            p[c / 2 + 1] = pack_half2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
          }
          tmem_st16(st + half / 2, p);  // over columns that have been read
        }
        l += (__uint_as_float(la[0]) + __uint_as_float(la[1])) + (__uint_as_float(la[2]) + __uint_as_float(la[3]));
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&sm->p_full[b]);
        issue_pv(i);
      }
      // ---- this segment's record
      ok = __all_sync(kFull, ok && wait(sm->pv_done, it + nt - 1));
      if (ok) {
        tc_fence_after();
        const size_t slot = size_t(ci + un.u);
        float4* rec = reinterpret_cast<float4*>(a.ws + sa.sl.off_rec) + (slot * kQ + v) * (kHeadDim / 4);
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 32) {
          uint32_t o[32];
          tmem_ld32(lanes + c, o);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            rec[(c + j) / 4] = make_float4(__uint_as_float(o[j]) + z, __uint_as_float(o[j + 1]) + z,
                                           __uint_as_float(o[j + 2]) + z, __uint_as_float(o[j + 3]) + z);
        }
        reinterpret_cast<float*>(a.ws + sa.sl.off_m)[slot * kQ + v] = m == kNegInf ? kNegInf : m - sg;
        reinterpret_cast<float*>(a.ws + sa.sl.off_l)[slot * kQ + v] = l;
        tc_fence_before();
      } else {
        give_up();
      }
    }
    it += nt;
    __syncthreads();  // Q, the lengths and O are free for the next segment
    if (sm->dead) break;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_free(tmem, kTmemCols);
}

template <int KB, int VB, bool ASYM>
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
    int sms = 0, room = 0;
    const auto k = shared_tc_kernel<KB, VB, ASYM>;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&room, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess ||
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes()) != cudaSuccess ||
        cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess)
      return 0;
    // two CTAs fit an SM: 128 registers a thread, 256 of 512 tensor-memory columns and the shared memory
    // (the occupancy query answers one for a kernel that uses tensor memory)
    return done[dev] = sms * (2 * (smem_bytes() + 1024) <= room ? 2 : 1);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, shared_tc_kernel<KB, VB, ASYM>, a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
  }
};

template <class F>
auto by_format(const CacheView& c, F f) {
  const int kb = c.k_bits, vb = c.v_bits;
  const bool as = c.asym != 0;
  if (kb == 8 && vb == 8) return as ? f(SharedTcKernel<8, 8, true>{}) : f(SharedTcKernel<8, 8, false>{});
  if (kb == 4 && vb == 4) return as ? f(SharedTcKernel<4, 4, true>{}) : f(SharedTcKernel<4, 4, false>{});
  if (kb == 4 && vb == 8) return as ? f(SharedTcKernel<4, 8, true>{}) : f(SharedTcKernel<4, 8, false>{});
  if (kb == 8 && vb == 4) return as ? f(SharedTcKernel<8, 4, true>{}) : f(SharedTcKernel<8, 4, false>{});
  return as ? f(SharedTcKernel<2, 2, true>{}) : f(SharedTcKernel<2, 2, false>{});
}

}  // namespace

int shared_tc_ctas(const CacheView& c) {
  return by_format(c, [](auto k) { return decltype(k)::ctas(); });
}

cudaError_t launch_shared_tc(const SharedArgs& a, cudaStream_t s) {
  return by_format(a.d.c, [&](auto k) { return decltype(k)::launch(a, s); });
}

}  // namespace kvq
