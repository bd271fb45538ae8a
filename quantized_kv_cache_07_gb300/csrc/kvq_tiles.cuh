// Query-tile device code shared by chunked prefill (kvq_prefill_tiles.cu) and
// shared-prefix decode (kvq_shared_tiles.cu): 16 query vectors meet one cached
// block on mma.sync, scores, online softmax and value product (the layout and
// the mathematics are described in kvq_prefill_tiles.cu).
#pragma once

#include "kvq_decode_impl.cuh"

namespace kvq {
namespace {

constexpr int kTileQ = 16;       // query vectors per tile: one m16 row tile
constexpr int kOStride = 132;    // float row stride of the combine buffer (bank spread)
constexpr float kFloatMax = 3.4028234663852886e38f;
constexpr int kCombineBytes = kConsumerWarps * kTileQ * kOStride * 4;

template <int KB, int VB, bool ASYM>
struct TileFmt {
  using F = Fmt<KB, VB, ASYM>;
  static constexpr int kBlocksPerStage = kConsumerWarps;  // block w of a stage -> consumer warp w
  static constexpr int kStageBytes = kBlocksPerStage * F::kPerBlock;
  static constexpr int kStagesRaw = 65536 / kStageBytes;
  static constexpr int kStages = kStagesRaw < 2 ? 2 : (kStagesRaw > 16 ? 16 : kStagesRaw);
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kBlocksPerStage * F::kKBB;
  static constexpr int kOffMeta = kOffV + kBlocksPerStage * F::kVBB;
  // the four warps' states merge in the ring once a sub-pass has drained it
  static_assert(kStages * kStageBytes >= kCombineBytes, "combine buffer must fit in the ring");
};

struct TileSmem {
  int qf, qlo, qs, qz, zo, qlen, cm, cl, rowseq, rowlen, bars, total;
};

__host__ __device__ constexpr int align16(int x) { return (x + 15) & ~15; }

__host__ __device__ inline TileSmem tile_smem(int ring_bytes, int stages) {
  TileSmem m{};
  int o = align16(ring_bytes);
  m.qf = o;  // query tile in A-operand order: [slice kk][g][t] x (rows g, g + 8) x 4 fp16
  o = align16(o + 8 * 8 * 4 * 16);
  m.qlo = o;  // two-part mode: the low fp16 parts in the same order
  o = align16(o + 8 * 8 * 4 * 16);
  m.qs = o;
  o = align16(o + kTileQ * 4);
  m.qz = o;  // asymmetric blocks: sum of each fp16 query vector as the MMA sees it
  o = align16(o + kTileQ * 4);
  m.zo = o;  // offset int8 keys: float4 per g {even g, even g + 8, odd g, odd g + 8}
  o = align16(o + kTileQ * 2 * 4);
  m.qlen = o;
  o = align16(o + kTileQ * 4);
  m.cm = o;
  o = align16(o + kConsumerWarps * kTileQ * 4);
  m.cl = o;
  o = align16(o + kConsumerWarps * kTileQ * 4);
  m.rowseq = o;
  o = align16(o + kTileQ * 4);
  m.rowlen = o;
  o = align16(o + kTileQ * 4);
  m.bars = o;
  o = align16(o + (2 * stages + 2) * 8);
  m.total = o;
  return m;
}

// Int8 keys of the one-part query modes enter the score product with their
// offset (s8x4_to_f16_r_off: 1152 + c, exact) and each block's accumulators
// start at minus 1152 times the row's sum over the dims they cover (the even
// k-slices for s, the odd ones for the second chain), as in the decode kernel.
template <int KB, bool LOQ>
struct TileOffsetKeys {
  static constexpr bool kOn = !LOQ && KB == 8;
};

// Four int8 codes -> (1152 + c0, 1152 + c1), (1152 + c2, 1152 + c3); c64 as below.
__device__ __forceinline__ void s8x4_to_f16_r_off(uint32_t w, uint32_t c64, uint32_t& lo, uint32_t& hi) {
  lo = __byte_perm(w, c64, 0x4140);
  hi = __byte_perm(w, c64, 0x4342);
}

// Four int8 codes -> fp16 pairs as s8x4_to_f16, with the byte constant 0x64
// of the permutes in a register (c64 = 0x64646464 from the caller) instead of
// being rebuilt before every permute.
__device__ __forceinline__ void s8x4_to_f16_r(uint32_t w, uint32_t c64, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(w, c64, 0x4140);
  const uint32_t b = __byte_perm(w, c64, 0x4342);
  const uint32_t bias = 0x64806480u;  // (1152, 1152) = 1024 + 128
  asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(bias));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(bias));
}

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Online-softmax state of one consumer warp over its blocks of a sub-pass:
// each thread holds rows g and g + 8 of the tile, output dims 8 nt + 2t, +1.
struct TileState {
  float O[16][4];
  float m0, m1, l0, l1;
  float z0, z1;     // asymmetric values: sum of p * m'_v of this thread's tokens per row
  float sg0, sg1;   // sigma of each row (as in decode), by the value scales that the row sees (one chunk: sg0 for both),
  float svlim;      // and the largest value scale that both allow
  __device__ __forceinline__ void reset() {
    m0 = m1 = kNegInf;
    l0 = l1 = 0.f;
    z0 = z1 = 0.f;
    sg0 = sg1 = float(kSigma0);
    svlim = ldexpf(1.f, kWeightExp - int(kMaxSlack) - kSigma0);
#pragma unroll
    for (int i = 0; i < 16; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.f;
  }
};

// Scores of one block: s[n][c] for n-tile n (tokens 8n..8n+7), row g (c < 2)
// or g + 8, token 8n + 2t + (c & 1).  Key slice kk covers dims 32t + 4kk + 0..3
// of every lane (the fragment-native key order); qf holds the query tile in
// the same order with rows g and g + 8 interleaved, so the A operand of slice
// kk is one 16-byte load, its four registers in operand order.
// With OFF the accumulators start at zi: {even row g, even row g + 8, odd row
// g, odd row g + 8} (TileOffsetKeys).
template <int KB, bool LOQ, bool OFF>
__device__ __forceinline__ void tile_scores(const uint8_t* kb, const uint4* qf, const uint4* qlo, float (&s)[2][4],
                                            int lane, uint32_t km, uint32_t c64, float4 zi) {
  auto qa = [&](int kk, uint32_t (&r)[4]) {
    const uint4 u = qf[kk * 32 + lane];
    r[0] = u.x;
    r[1] = u.y;
    r[2] = u.z;
    r[3] = u.w;
  };
  // one slice's product for n-tile d: the high query parts, then (two-part
  // mode) the low parts into the same accumulator
  auto mma2 = [&](float (&d)[4], int kk, const uint32_t (&q)[4], uint32_t b0, uint32_t b1) {
    if constexpr (KB == 16) {
      mma_bf16(d, q[0], q[1], q[2], q[3], b0, b1);
      return;
    }
    mma_f16(d, q[0], q[1], q[2], q[3], b0, b1);
    if constexpr (LOQ) {
      const uint4 l = qlo[kk * 32 + lane];
      mma_f16(d, l.x, l.y, l.z, l.w, b0, b1);
    }
  };
  float e[2][4];  // odd slices: a second chain
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    s[n][0] = s[n][1] = OFF ? zi.x : 0.f;
    s[n][2] = s[n][3] = OFF ? zi.y : 0.f;
    e[n][0] = e[n][1] = OFF ? zi.z : 0.f;
    e[n][2] = e[n][3] = OFF ? zi.w : 0.f;
  }
  const uint4* p = reinterpret_cast<const uint4*>(kb) + lane;
  if constexpr (KB == 8) {
    const uint4 r0a = p[0], r0b = p[32], r1a = p[64], r1b = p[96];
    const uint32_t g0[8] = {r0a.x, r0a.y, r0a.z, r0a.w, r0b.x, r0b.y, r0b.z, r0b.w};
    const uint32_t g8[8] = {r1a.x, r1a.y, r1a.z, r1a.w, r1b.x, r1b.y, r1b.z, r1b.w};
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      uint32_t a0, a1, a2, a3, q[4];
      qa(kk, q);
      if constexpr (OFF) {
        s8x4_to_f16_r_off(g0[kk], c64, a0, a2);  // tokens 0-7
        s8x4_to_f16_r_off(g8[kk], c64, a1, a3);  // tokens 8-15
      } else {
        s8x4_to_f16_r(g0[kk], c64, a0, a2);
        s8x4_to_f16_r(g8[kk], c64, a1, a3);
      }
      float(&d)[2][4] = (kk & 1) ? e : s;
      mma2(d[0], kk, q, a0, a2);
      mma2(d[1], kk, q, a1, a3);
    }
  } else if constexpr (KB == 2) {
    // one 16-byte load: word w holds slices 2w (outputs 0-3) and 2w+1 (4-7),
    // outputs (token g, token g+8) x (dims +0,+1 and +2,+3) of the slice
    const uint4 r = p[0];
    const uint32_t wd[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int wi = 0; wi < 4; ++wi) {
      uint32_t o[8], q0[4], q1[4];
      s2x16_to_f16(wd[wi], km, o);
      qa(2 * wi, q0);
      qa(2 * wi + 1, q1);
      mma2(s[0], 2 * wi, q0, o[0], o[2]);
      mma2(s[1], 2 * wi, q0, o[1], o[3]);
      mma2(e[0], 2 * wi + 1, q1, o[4], o[6]);
      mma2(e[1], 2 * wi + 1, q1, o[5], o[7]);
    }
  } else if constexpr (KB == 16) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const uint4 lo = p[(kk >> 1) * 32], hi = p[(4 + (kk >> 1)) * 32];  // tokens 0-7, 8-15
      uint32_t q[4];
      qa(kk, q);
      float(&d)[2][4] = (kk & 1) ? e : s;
      mma2(d[0], kk, q, (kk & 1) ? lo.z : lo.x, (kk & 1) ? lo.w : lo.y);
      mma2(d[1], kk, q, (kk & 1) ? hi.z : hi.x, (kk & 1) ? hi.w : hi.y);
    }
  } else {
    const uint4 r0 = p[0], r1 = p[32];
    const uint32_t g0[4] = {r0.x, r0.y, r0.z, r0.w};
    const uint32_t g8[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int wi = 0; wi < 4; ++wi) {
      uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
      s4x8_to_f16(g0[wi], km, x0, x1, x2, x3);
      s4x8_to_f16(g8[wi], km, y0, y1, y2, y3);
      uint32_t q0[4], q1[4];
      qa(2 * wi, q0);
      qa(2 * wi + 1, q1);
      mma2(s[0], 2 * wi, q0, x0, x1);
      mma2(s[1], 2 * wi, q0, y0, y1);
      mma2(e[0], 2 * wi + 1, q1, x2, x3);
      mma2(e[1], 2 * wi + 1, q1, y2, y3);
    }
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[n][c] += e[n][c];
}

// O += P . V for one block: P in A-operand registers (rows g / g + 8, token
// slots in the value block's order), V codes converted to the B-operand pairs
// of dims 16 mt + g (O[2 mt]) and 16 mt + 8 + g (O[2 mt + 1]).
template <int VB, bool LOW>
__device__ __forceinline__ void tile_values(const uint8_t* vb, const uint32_t (&ph)[4], const uint32_t (&pl)[4],
                                            float (&O)[16][4], int lane, uint32_t km, uint32_t c64, int valid,
                                            int head, int from) {
  const uint4* p = reinterpret_cast<const uint4*>(vb) + lane;
  // the high weights, then (two-part mode) the low weights into the same accumulator
  auto mma2 = [&](float (&d)[4], uint32_t b0, uint32_t b1) {
    if constexpr (VB == 16) {  // bf16 weights, always in two parts
      mma_bf16(d, ph[0], ph[1], ph[2], ph[3], b0, b1);
      mma_bf16(d, pl[0], pl[1], pl[2], pl[3], b0, b1);
      return;
    }
    mma_f16(d, ph[0], ph[1], ph[2], ph[3], b0, b1);
    if constexpr (LOW) mma_f16(d, pl[0], pl[1], pl[2], pl[3], b0, b1);
  };
  if constexpr (VB == 8) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const uint4 c = p[h * 32];
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};  // (mt 2h, dims lo), (2h, hi), (2h+1, lo), (2h+1, hi)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t b0, b1;
        s8x4_to_f16_r(w[k], c64, b0, b1);
        mma2(O[4 * h + k], b0, b1);
      }
    }
  } else if constexpr (VB == 2) {
    // one 16-byte load: word w holds m-tiles 2w (outputs 0-3) and 2w+1 (4-7)
    const uint4 c = p[0];
    const uint32_t wd[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int wi = 0; wi < 4; ++wi) {
      uint32_t o[8];
      s2x16_to_f16(wd[wi], km, o);
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // m-tile 2 wi + h
        mma2(O[2 * (2 * wi + h)], o[4 * h], o[4 * h + 2]);
        mma2(O[2 * (2 * wi + h) + 1], o[4 * h + 1], o[4 * h + 3]);
      }
    }
  } else if constexpr (VB == 16) {
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      uint4 c = p[mt * 32];  // dims lo (x, y), dims hi (z, w): token pairs of the two slot halves
      if (valid < kBlock || (from > 0 && head < kBlock)) {  // slots that no row sees are not data
        const uint32_t even = bf16_data(lane, 0, valid, head, from), odd = bf16_data(lane, 1, valid, head, from);
        c = make_uint4(c.x & even, c.y & odd, c.z & even, c.w & odd);
      }
      mma2(O[2 * mt], c.x, c.y);
      mma2(O[2 * mt + 1], c.z, c.w);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 c = p[h * 32];
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // m-tile 4h + k
        uint32_t x0, x1, x2, x3;
        s4x8_to_f16(w[k], km, x0, x1, x2, x3);
        mma2(O[2 * (4 * h + k)], x0, x1);
        mma2(O[2 * (4 * h + k) + 1], x2, x3);
      }
    }
  }
}

// One block of one consumer warp: scores, causal mask, online softmax with the
// lazy maximum and the sigma offset of the decode kernel, value product.
// APART: the rows are those of different sequences, and a value scale that is out of the others' range, or not
// finite, counts in the rows that see its token alone; otherwise (rows of one chunk) one sigma serves both
// rows (separate ones cost the chunked prefill 1.7 %: 201.0 us for 197.6; the shared prefix of 4 sequences of 2048
// tokens 2 %, 21.8 us and 22.3).
// SPAN: row r sees tokens below ts.sinks and from its length - ts.span on; none of the rows sees those between
// ts.sinks and ts.from.
struct TileSpan {
  int sinks, span, from;
};
template <int KB, int VB, bool ASYM, bool LOQ, bool APART, bool SPAN = false>
__device__ __forceinline__ void tile_block(const uint8_t* kb, const uint8_t* vb, const float* ks, const float* vs,
                                           const float* ko, const float* vo, int tok0, int maxlen, int len0,
                                           int len1, float qs0, float qs1, float qz0, float qz1, const uint4* qf,
                                           const uint4* qlo, const float4* zo, TileState& st, int lane, uint32_t km,
                                           uint32_t c64, const TileSpan& ts = TileSpan{}) {
  // does a row of this length, and does any row, see the token at pos
  auto sees = [&](int pos, int len) { return pos < len && (!SPAN || pos < ts.sinks || pos >= len - ts.span); };
  auto seen = [&](int pos) { return pos < maxlen && (!SPAN || pos < ts.sinks || pos >= ts.from); };
  // offset-binary centre of the code conversion: c' = u - kKC (zero points: m' = m + kKC * s)
  constexpr float kKC = KB == 8 ? 128.f : (KB == 4 ? 8.f : 2.f), kVC = VB == 8 ? 128.f : (VB == 4 ? 8.f : 2.f);
  // 2-bit blocks: one scale (and zero point) for the whole block
  constexpr bool kGroup = KB == 2;
  const int t = lane & 3;
  float x[2][4];
  constexpr bool kOff = TileOffsetKeys<KB, LOQ>::kOn;
  tile_scores<KB, LOQ, kOff>(kb, qf, qlo, x, lane, km, c64, kOff ? zo[lane >> 2] : make_float4(0.f, 0.f, 0.f, 0.f));
  constexpr bool kBf16 = KB == 16;
  const float2 one = make_float2(1.f, 1.f);
  // this thread's tokens: 8n + 2t + j (n = 0, 1; j = 0, 1)
  const float2 k0 = kBf16 ? one : kGroup ? make_float2(ks[0], ks[0]) : *reinterpret_cast<const float2*>(ks + 2 * t);
  const float2 k1 = kBf16 ? one : kGroup ? make_float2(ks[0], ks[0]) : *reinterpret_cast<const float2*>(ks + 8 + 2 * t);
  const float2 v0 = kBf16 ? one : kGroup ? make_float2(vs[0], vs[0]) : *reinterpret_cast<const float2*>(vs + 2 * t);
  const float2 v1 = kBf16 ? one : kGroup ? make_float2(vs[0], vs[0]) : *reinterpret_cast<const float2*>(vs + 8 + 2 * t);
  const float ksc[2][2] = {{k0.x, k0.y}, {k1.x, k1.y}};
  float vsc[2][2] = {{v0.x, v0.y}, {v1.x, v1.y}};
  float mk[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, mv[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
  if constexpr (ASYM) {
    const float2 a0 = kGroup ? make_float2(ko[0], ko[0]) : *reinterpret_cast<const float2*>(ko + 2 * t);
    const float2 a1 = kGroup ? make_float2(ko[0], ko[0]) : *reinterpret_cast<const float2*>(ko + 8 + 2 * t);
    const float2 b0 = kGroup ? make_float2(vo[0], vo[0]) : *reinterpret_cast<const float2*>(vo + 2 * t);
    const float2 b1 = kGroup ? make_float2(vo[0], vo[0]) : *reinterpret_cast<const float2*>(vo + 8 + 2 * t);
    mk[0][0] = fmaf(kKC, k0.x, a0.x);
    mk[0][1] = fmaf(kKC, k0.y, a0.y);
    mk[1][0] = fmaf(kKC, k1.x, a1.x);
    mk[1][1] = fmaf(kKC, k1.y, a1.y);
    mv[0][0] = fmaf(kVC, v0.x, b0.x);
    mv[0][1] = fmaf(kVC, v0.y, b0.y);
    mv[1][0] = fmaf(kVC, v1.x, b1.x);
    mv[1][1] = fmaf(kVC, v1.y, b1.y);
  }
  float svm = 0.f;
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int pos = tok0 + 8 * n + 2 * t + j;
      if constexpr (ASYM) {
        x[n][j] = sees(pos, len0) ? fmaf(x[n][j], ksc[n][j], mk[n][j] * qz0) * qs0 : kNegInf;
        x[n][2 + j] = sees(pos, len1) ? fmaf(x[n][2 + j], ksc[n][j], mk[n][j] * qz1) * qs1 : kNegInf;
        mv[n][j] = seen(pos) ? mv[n][j] : 0.f;
      } else {
        x[n][j] = sees(pos, len0) ? x[n][j] * (ksc[n][j] * qs0) : kNegInf;
        x[n][2 + j] = sees(pos, len1) ? x[n][2 + j] * (ksc[n][j] * qs1) : kNegInf;
      }
      // scales of slots past the sub-pass's longest row are not data
      vsc[n][j] = seen(pos) ? vsc[n][j] : 0.f;
      svm = APART ? max_nan(svm, vsc[n][j]) : fmaxf(svm, vsc[n][j]);
    }
  float mx0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
  float mx1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {  // the four lanes of a row
    mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, o));
    mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, o));
  }
  if (__any_sync(kFull, (mx0 > st.m0 + kMaxSlack) || (mx1 > st.m1 + kMaxSlack))) {
    const float mn0 = fmaxf(st.m0, mx0), mn1 = fmaxf(st.m1, mx1);
    const float al0 = (mn0 == kNegInf) ? 1.f : ex2(st.m0 - mn0);
    const float al1 = (mn1 == kNegInf) ? 1.f : ex2(st.m1 - mn1);
    st.l0 *= al0;
    st.l1 *= al1;
    st.z0 *= al0;
    st.z1 *= al1;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      st.O[i][0] *= al0;
      st.O[i][1] *= al0;
      st.O[i][2] *= al1;
      st.O[i][3] *= al1;
    }
    st.m0 = mn0;
    st.m1 = mn1;
  }
  if (__any_sync(kFull, APART ? !(svm <= st.svlim) : svm > st.svlim)) {
    int sn0, sn1;
    float q0 = 1.f, q1 = 1.f;  // not a number for a row whose outputs are none
    if constexpr (APART) {
      // Each row by the scales that it sees: a token of one sequence leaves the others alone.  One whose scale is not
      // finite makes the outputs of the rows that see it no number, and then counts as 0 (a hidden one would be 0 x inf).
      float s0 = 0.f, s1 = 0.f;
      bool bad0 = false, bad1 = false;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int pos = tok0 + 8 * n + 2 * t + j;
          const bool in0 = sees(pos, len0), in1 = sees(pos, len1);
          if (!(vsc[n][j] <= kFloatMax)) {
            bad0 |= in0;
            bad1 |= in1;
            vsc[n][j] = mv[n][j] = 0.f;
          }
          s0 = in0 ? fmaxf(s0, vsc[n][j]) : s0;
          s1 = in1 ? fmaxf(s1, vsc[n][j]) : s1;
        }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        s0 = fmaxf(s0, __shfl_xor_sync(kFull, s0, o));
        s1 = fmaxf(s1, __shfl_xor_sync(kFull, s1, o));
      }
      const unsigned row = 0xFu << (lane & ~3);  // the four lanes of the rows
      q0 = __ballot_sync(kFull, bad0) & row ? __int_as_float(0x7fffffff) : 1.f;
      q1 = __ballot_sync(kFull, bad1) & row ? __int_as_float(0x7fffffff) : 1.f;
      int e0, e1;
      frexpf(s0, &e0);  // s0 < 2^e0
      frexpf(s1, &e1);
      sn0 = s0 > 0.f ? min(int(st.sg0), kWeightExp - int(kMaxSlack) - e0) : int(st.sg0);
      sn1 = s1 > 0.f ? min(int(st.sg1), kWeightExp - int(kMaxSlack) - e1) : int(st.sg1);
    } else {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) svm = fmaxf(svm, __shfl_xor_sync(kFull, svm, o));
      int ex;
      frexpf(svm, &ex);  // svm < 2^ex
      sn0 = sn1 = min(int(st.sg0), kWeightExp - int(kMaxSlack) - ex);
    }
    const float f0 = ldexpf(1.f, sn0 - int(st.sg0)), f1 = APART ? ldexpf(1.f, sn1 - int(st.sg1)) : f0;  // exact powers of two
    st.l0 *= f0;
    st.l1 *= f1;
    st.z0 *= f0;
    st.z1 *= f1;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      st.O[i][0] *= APART ? f0 * q0 : f0;
      st.O[i][1] *= APART ? f0 * q0 : f0;
      st.O[i][2] *= APART ? f1 * q1 : f1;
      st.O[i][3] *= APART ? f1 * q1 : f1;
    }
    st.sg0 = float(sn0);
    st.sg1 = float(sn1);
    // rows that have ended, or were never there, have no more say
    const int top = APART ? max(tok0 < len0 ? sn0 : -256, tok0 < len1 ? sn1 : -256) : sn0;
    st.svlim = top == -256 ? kFloatMax : ldexpf(1.f, kWeightExp - int(kMaxSlack) - top);
  }
  const float base0 = (st.m0 == kNegInf) ? 0.f : st.m0 - st.sg0;
  const float base1 = (st.m1 == kNegInf) ? 0.f : st.m1 - (APART ? st.sg1 : st.sg0);
  float w[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float pa = ex2(x[n][j] - base0), pb = ex2(x[n][2 + j] - base1);
      st.l0 += pa;
      st.l1 += pb;
      if constexpr (ASYM) {
        st.z0 = fmaf(pa, mv[n][j], st.z0);
        st.z1 = fmaf(pb, mv[n][j], st.z1);
      }
      w[n][j] = pa * vsc[n][j];
      w[n][2 + j] = pb * vsc[n][j];
    }
  // A operand of the value product: token slot k of the value block order
  // holds tokens (2t, 2t + 8) at k = (2t, 2t + 1) and (2t + 1, 2t + 9) at
  // k = (2t + 8, 2t + 9)
  const float wr[4][2] = {{w[0][0], w[1][0]}, {w[0][2], w[1][2]}, {w[0][1], w[1][1]}, {w[0][3], w[1][3]}};
  uint32_t ph[4], pl[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // registers: row g, row g + 8, row g, row g + 8
    if constexpr (kBf16) {
      ph[i] = pack_bf162(wr[i][0], wr[i][1]);
      pl[i] = pack_bf162(wr[i][0] - __uint_as_float(ph[i] << 16), wr[i][1] - __uint_as_float(ph[i] & 0xFFFF0000u));
      continue;
    }
    ph[i] = pack_half2(wr[i][0], wr[i][1]);
    if constexpr (LOQ) {  // low parts w - hi (exact in fp32)
      const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&ph[i]));
      pl[i] = pack_half2(wr[i][0] - hf.x, wr[i][1] - hf.y);
    }
  }
  tile_values<VB, LOQ>(vb, ph, pl, st.O, lane, km, c64, maxlen - tok0, SPAN ? ts.sinks - tok0 : kBlock,
                       SPAN ? ts.from - tok0 : 0);
}

// Query vector v of a tile (src: its 128 bf16 values, or null for an unused
// one) into the A-operand order of the tile, by one warp; returns its score
// scale.  Code blocks: fp16 scaled by a power of two per vector (the decode
// kernel's query format), or int8 codes (q_bits 8), with the low parts of the
// two-part mode, the zero-point sums and the offset terms beside it.
template <int KB, bool ASYM, bool LOQ>
__device__ __forceinline__ float stage_tile_vector(const DecodeArgs& a, const uint16_t* src, int h, int v, uint32_t* qf,
                                                   uint32_t* qlo, float* qz_s, float* zo_s, int lane) {
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (src) {
    const uint2 raw = __ldcg(reinterpret_cast<const uint2*>(src + 4 * lane));
    x[0] = __uint_as_float(raw.x << 16);
    x[1] = __uint_as_float(raw.x & 0xFFFF0000u);
    x[2] = __uint_as_float(raw.y << 16);
    x[3] = __uint_as_float(raw.y & 0xFFFF0000u);
    if (a.c.factor) {
      const float4 c = __ldcg(reinterpret_cast<const float4*>(a.c.factor + h * kHeadDim + 4 * lane));
      x[0] *= c.x;
      x[1] *= c.y;
      x[2] *= c.z;
      x[3] *= c.w;
    }
  }
  if constexpr (KB == 16) {  // bf16 blocks: the query as it is
    const int at = (((lane & 7) * 8 + (v & 7)) * 4 + (lane >> 3)) * 4 + (v >> 3);
    qf[at] = pack_bf162(x[0], x[1]);
    qf[at + 2] = pack_bf162(x[2], x[3]);
    return kLog2e * kInvSqrtD;
  }
  float am = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(kFull, am, o));
  uint2 packed;
  float ylo[4] = {0.f, 0.f, 0.f, 0.f};  // the scaled fp32 values (two-part mode: their low parts)
  float qscale;  // score scale of the vector: log2(e) / sqrt(D) over its fp16 scaling
  if (a.c.q_bits == 8) {
    // int8 query rows: codes (exact in fp16) with the row scale s_q folded
    // into the score scale; the MMA then forms the integer dot exactly
    float cq[4];
    const float sq = quantize_int8_row(x, am, cq);
    packed.x = pack_half2(cq[0], cq[1]);
    packed.y = pack_half2(cq[2], cq[3]);
    qscale = sq * (kLog2e * kInvSqrtD);
  } else {
    int e = 0;
    if (am > 0.f) {
      int ex;
      frexpf(am, &ex);
      e = 15 - ex;  // am * 2^e in [2^14, 2^15)
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) ylo[j] = ldexpf(x[j], e);
    packed.x = pack_half2(ylo[0], ylo[1]);
    packed.y = pack_half2(ylo[2], ylo[3]);
    qscale = ldexpf(kLog2e * kInvSqrtD, -e);
  }
  if constexpr (ASYM) {  // the vector's sum exactly as the MMA sees it
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&packed.x));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&packed.y));
    float z = (f0.x + f0.y) + (f1.x + f1.y);
    if constexpr (LOQ) {  // plus the low parts, as the second product sees them
      const uint32_t l0 = pack_half2(ylo[0] - f0.x, ylo[1] - f0.y), l1 = pack_half2(ylo[2] - f1.x, ylo[3] - f1.y);
      const float2 g0 = __half22float2(*reinterpret_cast<const __half2*>(&l0));
      const float2 g1 = __half22float2(*reinterpret_cast<const __half2*>(&l1));
      z += (g0.x + g0.y) + (g1.x + g1.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
    if (lane == 0) qz_s[v] = z;
  }
  if constexpr (TileOffsetKeys<KB, LOQ>::kOn) {
    // offset terms: minus 1152 times the vector's sums over the even and
    // the odd k-slices (this lane's dims 4 lane .. +3 lie in slice lane & 7)
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&packed.x));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&packed.y));
    float zs = (f0.x + f0.y) + (f1.x + f1.y);
#pragma unroll
    for (int o = 16; o > 1; o >>= 1) zs += __shfl_xor_sync(kFull, zs, o);
    if (lane < 2) zo_s[(v & 7) * 4 + 2 * lane + (v >> 3)] = -kOffsetF16 * zs;
  }
  {  // dims 4 lane .. +3 = 32t + 4kk + 0..3 of vector v = row g (+ 8)
    const int at = (((lane & 7) * 8 + (v & 7)) * 4 + (lane >> 3)) * 4 + (v >> 3);
    qf[at] = packed.x;
    qf[at + 2] = packed.y;
    if constexpr (LOQ) {  // two-part query: the low parts y - hi (exact in fp32)
      const float2 h0 = __half22float2(*reinterpret_cast<const __half2*>(&packed.x));
      const float2 h1 = __half22float2(*reinterpret_cast<const __half2*>(&packed.y));
      qlo[at] = pack_half2(ylo[0] - h0.x, ylo[1] - h0.y);
      qlo[at + 2] = pack_half2(ylo[2] - h1.x, ylo[3] - h1.y);
    }
  }
  return qscale;
}

}  // namespace
}  // namespace kvq
