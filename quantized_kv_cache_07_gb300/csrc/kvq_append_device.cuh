// Device code of the quantizing write, shared by kvq_append (kvq_append.cu) and
// the rotary write (kvq_rope.cu): the per-vector quantizers, the stores into a
// block, the window ring, and the whole-block write of 2-bit caches.
#pragma once

#include "kvq_device.cuh"
#include "kvq_launch.h"

namespace kvq {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float bf16_bits_to_f32(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

// Warp-cooperative per-vector quantization.
__device__ __forceinline__ void quantize_warp(const float (&x)[4], int bits, int (&code)[4], float& s) {
  // non-negative floats order as their bits: one warp reduction; NaN counts as the least
  const float own = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
  const float a = __int_as_float(__reduce_max_sync(kFull, own != own ? -1 : __float_as_int(own)));
  if (a == 0.0f) {
    s = 1.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) code[j] = 0;
    return;
  }
  s = __fdiv_rn(a, bits == 8 ? 127.f : 7.f);
  round_quotients(x, s, __frcp_rn(s), bits == 8 ? -127 : -8, bits == 8 ? 127 : 7, code);
}

// Warp-cooperative asymmetric quantization: m = min(x), s = RN32((max - min) /
// (2^bits - 1)) with the difference and the quotient in double (a constant
// vector gets s = 1), u = clamp(rint((x - m) / s), 0, 2^bits - 1) with the
// difference and the quotient in double (rint: half to even).
__device__ __forceinline__ void quantize_asym_warp(const float (&x)[4], int bits, int (&u)[4], float& s, float& m) {
  float lo = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
  float hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
  }
  const int qmaxu = bits == 8 ? 255 : 15;
  const double rng = __dsub_rn(double(hi), double(lo));
  s = rng == 0.0 ? 1.0f : __double2float_rn(__ddiv_rn(rng, double(qmaxu)));
  m = lo;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const double r = rint(__ddiv_rn(__dsub_rn(double(x[j]), double(lo)), double(s)));
    u[j] = r >= double(qmaxu) ? qmaxu : (r > 0.0 ? int(r) : 0);  // clamp before the conversion
  }
}

// The asymmetric quantizer out of line (its divisions in double are long code).
struct AsymCodes {
  int u[4];
  float s, m;
};
static __device__ __noinline__ AsymCodes quantize_asym_far(float4 v, int bits) {
  const float x[4] = {v.x, v.y, v.z, v.w};
  AsymCodes r;
  quantize_asym_warp(x, bits, r.u, r.s, r.m);
  return r;
}

// Store the codes of one quantized vector (token `tok`) into its block.  The
// values given are the stored bytes / nibbles (offset-binary for symmetric
// codes, the unsigned code itself for the asymmetric format).
__device__ void store_codes(bool is_key, int bits, uint8_t* blk, int tok, const int (&code)[4], int lane) {
  if (bits == 8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = 4 * lane + j;
      const Loc L = is_key ? key_loc(8, tok, d) : value_loc(8, tok, d);
      blk[L.byte] = uint8_t(code[j]);
    }
    return;
  }
  // 4-bit
  if (is_key) {
    // Lanes l and l^1 own the 8 nibbles of one 32-bit word of this token.
    uint32_t part = 0;
    int word_off = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = 4 * lane + j;
      const Loc L = key_loc(4, tok, d);
      const int nib = ((L.byte & 3) << 1) | (L.shift >> 2);
      part |= uint32_t(code[j]) << (4 * nib);
      word_off = L.byte & ~3;
    }
    const uint32_t word = part | __shfl_xor_sync(kFull, part, 1);
    if ((lane & 1) == 0) *reinterpret_cast<uint32_t*>(blk + word_off) = word;
    return;
  }
  // 4-bit values: a word mixes four tokens, so update only this token's nibbles.
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int d = 4 * lane + j;
    const Loc L = value_loc(4, tok, d);
    const int nib = ((L.byte & 3) << 1) | (L.shift >> 2);
    uint32_t* w = reinterpret_cast<uint32_t*>(blk + (L.byte & ~3));
    atomicAnd(w, ~(0xFu << (4 * nib)));
    atomicOr(w, uint32_t(code[j]) << (4 * nib));
  }
}

__device__ void store_bf16(bool is_key, uint8_t* blk, int tok, const uint16_t (&xb)[4], int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int d = 4 * lane + j;
    const Loc L = is_key ? key_loc(16, tok, d) : value_loc(16, tok, d);
    *reinterpret_cast<uint16_t*>(blk + L.byte) = xb[j];
  }
}

// Quantize (or copy, for a bf16 cache) one vector into the block store at
// position p of sequence b.
__device__ void write_block_store(const AppendArgs& a, bool is_key, int b, int p, int h, const uint16_t (&xb)[4],
                                  int lane) {
  const CacheView& c = a.c;
  if (p / kBlock >= a.mbps) {  // (in blocks: neither side passes 32 bits)
    if (lane == 0) flag(a.err, KVQ_DEVERR_POSITION);
    return;
  }
  const int phys = a.table[size_t(b) * a.mbps + p / kBlock];
  if (phys < 0 || phys >= c.num_blocks) {
    if (lane == 0) flag(a.err, KVQ_DEVERR_BLOCK_ID);
    return;
  }
  const int tok = p % kBlock;
  const int bits = is_key ? c.k_bits : c.v_bits;
  uint8_t* pool = is_key ? c.k_codes : c.v_codes;
  uint8_t* blk = pool + (size_t(h) * c.num_blocks + phys) * block_bytes(bits);
  if (bits == 16) {
    store_bf16(is_key, blk, tok, xb, lane);
    return;
  }
  float x[4];
  if (is_key && c.k_chan) {
    // per-channel scales only: code = clamp(rint(k / c)) of the exact quotient, no per-token scale
    const int lo = bits == 8 ? -127 : -8, hi = bits == 8 ? 127 : 7, bias = bits == 8 ? 128 : 8;
    int code[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float q = round_quotient(bf16_bits_to_f32(xb[j]), c.factor[h * kHeadDim + 4 * lane + j]);
      code[j] = int(fminf(float(hi), fmaxf(float(lo), q))) + bias;
    }
    store_codes(is_key, bits, blk, tok, code, lane);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = bf16_bits_to_f32(xb[j]);
    if (is_key && c.factor) x[j] = __fdiv_rn(x[j], c.factor[h * kHeadDim + 4 * lane + j]);
  }
  int code[4];
  float s, m = 0.f;
  const bool asym = c.asym != 0;
  if (asym) {
    quantize_asym_warp(x, bits, code, s, m);
  } else {
    quantize_warp(x, bits, code, s);
    const int bias = bits == 8 ? 128 : 8;  // offset binary
#pragma unroll
    for (int j = 0; j < 4; ++j) code[j] += bias;
  }
  store_codes(is_key, bits, blk, tok, code, lane);
  if (lane == 0) {
    // metadata record: K scales, (K zero points,) V scales, (V zero points)
    float* rec = c.meta + (size_t(h) * c.num_blocks + phys) * c.meta_floats;
    const int off = is_key ? 0 : c.meta_floats / 2;
    rec[off + tok] = s;
    if (asym) rec[off + kBlock + tok] = m;
  }
}

// Write one bf16 vector (lane l: dims 4l..4l+3 in xb) of sequence b, position p,
// head h: into the block store, or into the window ring (in KVQ_APPEND_STEP
// mode the token that leaves the ring is quantized into the block store first).
__device__ __forceinline__ void append_vector(const AppendArgs& a, bool is_key, int b, int p, int h,
                                              const uint16_t (&xb)[4], int lane) {
  if (a.mode == KVQ_APPEND_QUANT) {
    write_block_store(a, is_key, b, p, h, xb, lane);
    return;
  }
  // window ring: slot p % W is token (slot % 16) of ring block slot / 16, stored
  // in the fragment-native bf16 block layout
  const int W = a.c.window;
  const int slot = p % W;
  uint8_t* ring = (is_key ? a.c.k_win : a.c.v_win) +
                  ((size_t(b) * a.c.H + h) * (W / kBlock) + slot / kBlock) * block_bytes(16);
  const int tok = slot % kBlock;
  int off[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Loc L = is_key ? key_loc(16, tok, 4 * lane + j) : value_loc(16, tok, 4 * lane + j);
    off[j] = L.byte;
  }
  if (a.mode == KVQ_APPEND_STEP && p >= W) {
    // the token at p - W occupies this ring slot: it leaves the window now
    uint16_t ob[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) ob[j] = *reinterpret_cast<const uint16_t*>(ring + off[j]);
    write_block_store(a, is_key, b, p - W, h, ob, lane);
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<uint16_t*>(ring + off[j]) = xb[j];
}

// 2-bit blocks: one warp per (group, head, K or V).  A group is the run of rows
// of one call that fills positions 16j, 16j + 1, ... (up to 16) of one
// sequence; the row at position 16j leads it.  A row whose position is not at
// a block start and is not part of such a run is flagged and skipped: 2-bit
// blocks are written whole, in one call.
constexpr int kGroupWarps = 8;

// `ok(row)` says whether a row may be part of a run; `load(row, x)` gives lane
// l's dims 4l..4l+3 of a row (before the key factor).
template <class Ok, class Load>
__device__ __forceinline__ void append_group(const AppendArgs& a, int r, bool is_key, int h, uint32_t* im, int lane,
                                             Ok ok, Load load) {
  const int b = a.seq_idx[r];
  const int p = a.pos[r];
  if (b < 0 || b >= a.batch || p < 0 || !ok(r)) {
    if (lane == 0) flag(a.err, KVQ_DEVERR_POSITION);
    return;
  }
  const int j = p % kBlock;
  if (j != 0) {
    // covered by the run led by row r - j?
    bool covered = r - j >= 0;
    for (int k = 0; covered && k < j; ++k) covered = a.seq_idx[r - j + k] == b && a.pos[r - j + k] == p - j + k && ok(r - j + k);
    if (!covered && lane == 0) flag(a.err, KVQ_DEVERR_POSITION);
    return;
  }
  int m = 1;
  while (m < kBlock && r + m < a.n && a.seq_idx[r + m] == b && a.pos[r + m] == p + m && ok(r + m)) ++m;
  if (p / kBlock >= a.mbps) {  // p is a block's first position
    if (lane == 0) flag(a.err, KVQ_DEVERR_POSITION);
    return;
  }
  const int phys = a.table[size_t(b) * a.mbps + p / kBlock];
  if (phys < 0 || phys >= a.c.num_blocks) {
    if (lane == 0) flag(a.err, KVQ_DEVERR_BLOCK_ID);
    return;
  }
  // the group's values, lane l holding dims 4l..4l+3 of each row
  float x[kBlock][4];
#pragma unroll
  for (int k = 0; k < kBlock; ++k) {
    if (k < m) {
      load(r + k, x[k]);
      if (is_key && a.c.factor) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k][e] = __fdiv_rn(x[k][e], a.c.factor[h * kHeadDim + 4 * lane + e]);
      }
    } else {
      x[k][0] = x[k][1] = x[k][2] = x[k][3] = 0.f;
    }
  }
  const bool asym = a.c.asym != 0;
  float s = 1.f, zp = 0.f;
  float lo = x[0][0], hi = x[0][0], am = 0.f;
#pragma unroll
  for (int k = 0; k < kBlock; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (k < m) {
        lo = fminf(lo, x[k][e]);
        hi = fmaxf(hi, x[k][e]);
        am = fmaxf(am, fabsf(x[k][e]));
      }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
    am = fmaxf(am, __shfl_xor_sync(kFull, am, o));
  }
  if (asym) {
    // asymmetric rule over the group: m = min, s = RN32((max - min) / 3) (1 for
    // a constant group), u = clamp(rint((x - m) / s), 0, 3), in double
    const double rng = __dsub_rn(double(hi), double(lo));
    s = rng == 0.0 ? 1.0f : __double2float_rn(__ddiv_rn(rng, 3.0));
    zp = lo;
  } else if (am > 0.f) {
    s = am;  // RN32(amax / qmax) with qmax = 1
  }
#pragma unroll
  for (int i = lane; i < kBlock * kHeadDim * 2 / 32; i += 32) im[i] = 0u;
  __syncwarp();
#pragma unroll
  for (int k = 0; k < kBlock; ++k) {
    if (k >= m) break;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int u;
      if (asym) {
        const double q = rint(__ddiv_rn(__dsub_rn(double(x[k][e]), double(lo)), double(s)));
        u = q >= 3.0 ? 3 : (q > 0.0 ? int(q) : 0);
      } else {
        const float q = am > 0.f ? round_quotient(x[k][e], s) : 0.f;
        u = int(fminf(1.f, fmaxf(-2.f, q))) + 2;  // offset binary
      }
      const Loc L = is_key ? key_loc(2, k, 4 * lane + e) : value_loc(2, k, 4 * lane + e);
      atomicOr(&im[L.byte >> 2], uint32_t(u) << (8 * (L.byte & 3) + L.shift));
    }
  }
  __syncwarp();
  uint8_t* blk = (is_key ? a.c.k_codes : a.c.v_codes) + (size_t(h) * a.c.num_blocks + phys) * block_bytes(2);
  reinterpret_cast<uint4*>(blk)[lane] = reinterpret_cast<const uint4*>(im)[lane];
  if (lane == 0) {
    float* rec = a.c.meta + (size_t(h) * a.c.num_blocks + phys) * a.c.meta_floats;
    rec[is_key ? 0 : 2] = s;
    rec[is_key ? 1 : 3] = zp;
  }
}

}  // namespace
}  // namespace kvq
