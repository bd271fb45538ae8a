// Tiles of 64 cached tokens on tcgen05, common to shared-prefix decode (kvq_shared_tc.cu) and the
// chunked prefill with sinks (kvq_sinks_tc.cu): the orders inside a tile, codes and queries into swizzled shared memory.
#pragma once

#include "kvq_tcgen05.cuh"
#include "kvq_tiles.cuh"

namespace kvq {
namespace {

constexpr int kQ = 128;         // query vectors of a softmax warpgroup
constexpr int kTok = 64;        // tokens of a tile
constexpr int kTcThreads = 512;
constexpr int kTmemCols = 512;  // O of warpgroup j: 128 j; its S buffers: 256 + 128 j, + 64
constexpr int kRing = 4;        // stages of converted tiles

struct TcStage {
  uint8_t k[2][kTok * 128];  // two halves of 64 dims
  uint8_t v[kHeadDim * 128];
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

// A query vector into the swizzled Q tile by 8 lanes: lane `sub` holds dims 16 sub .. + 15 (raw: their bf16 bits,
// f: their key factors, if the cache has them).  The vector's score scale and sum (as the product sees it) come back.
// Four vectors a step in a loop, not unrolled: code that runs once is fetched at memory speed (unrolled over the
// 32 vectors of a warp the staging took 13 us).
// TWO: what the fp16 rounding leaves goes to a second tile `lo` bytes behind.
// FIXED: vectors of ordinary size (their largest value 2^-16 to 250, or zeros) are all scaled by 2^kFixedExp, exact in fp16
// for bf16 values from 2^-22 on; the scale that comes back is relative to that one's, 1 for them.
constexpr int kFixedExp = 8;
constexpr float kFixedLeast = 1.52587890625e-05f, kFixedMost = 250.f;
template <bool ASYM, bool TWO, bool FIXED = false>
__device__ __forceinline__ void put_query(const DecodeArgs& a, const uint4 (&raw)[2], const float (&f)[16], uint8_t* half,
                                          int lo, int row, int sub, float& scale, float& sum) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
      x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
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
  scale = kLog2e * kInvSqrtD;
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
    scale = FIXED ? s * float(1 << kFixedExp) : scale * s;
  } else {
    // exact powers of two: am * 2^(14 - e) in [2^14, 2^15); below 2^-112 the scores are zero to any precision
    const uint32_t e = max(__float_as_uint(am) >> 23, 15u);
    const bool fixed = FIXED && am <= kFixedMost && (am >= kFixedLeast || am == 0.f);
    const float f2 = fixed ? float(1 << kFixedExp) : __uint_as_float((268u - e) << 23);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] *= f2;
    if constexpr (FIXED) scale = fixed ? 1.f : __uint_as_float((e - 14u) << 23) * float(1 << kFixedExp);
    else scale *= __uint_as_float((e - 14u) << 23);
  }
  scale = fmaxf(scale, 1.17549435e-38f);  // positive, so that a masked score stays -inf
  sum = 0.f;
  const int t = sub >> 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // dims 32 t + 8 (2 (sub & 1) + i) ..: chunk i of this half
    uint32_t y[4], z[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x0 = x[8 * i + 2 * k], x1 = x[8 * i + 2 * k + 1];
      y[k] = pack_half2(x0, x1);
      if constexpr (ASYM || TWO) {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&y[k]));
        sum += h.x + h.y;
        if constexpr (TWO) {
          z[k] = pack_half2(x0 - h.x, x1 - h.y);
          const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&z[k]));
          sum += r.x + r.y;
        }
      }
    }
    uint4* const at = reinterpret_cast<uint4*>(half + row * 128 + ((dim_chunk(t, i) ^ (row & 7)) * 16));
    *at = make_uint4(y[0], y[1], y[2], y[3]);
    if constexpr (TWO) *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(at) + lo) = make_uint4(z[0], z[1], z[2], z[3]);
  }
  if constexpr (ASYM) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

}  // namespace
}  // namespace kvq
