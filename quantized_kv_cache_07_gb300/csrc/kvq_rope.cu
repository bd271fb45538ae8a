// Rotary positions with the cache write: kvq_rope_table and kvq_rope_append.
//
// A head's first R = rotary_dim dimensions are R / 2 pairs (x0, x1); at position
// p the pair j turns by the angle p * f_j:
//   y0 = x0 cos - x1 sin,  y1 = x0 sin + x1 cos,
// with pairs (j, j + R/2) (half layout) or (2j, 2j + 1) (interleaved).  Cosines
// and sines come from a float32 table [position][pair][2] that kvq_rope_table
// fills from angles in double: at position 10^5 a float32 angle would already
// be off by 4e-3.
//
// Rounding.  y is the exact value rounded to float32 (up to one case in about 2^24) and then to bf16.
// That makes the stored codes those of kvq_append on the rotated vectors bit for bit: a plain
// float32 sum differs from the exact one in its last bit often enough to move a bf16 rounding, with it
// a vector's largest value, and with that a whole vector's codes.  The sum with all its rounding errors (the
// products' by fused multiply-adds, the sum's by Knuth's two-sum) is 14
// instructions a value; a float32 sum with a bound on its error is 7 and decides all but one value in 10^4.
//
// One warp turns and writes one 128-element vector; lane l owns dims 4l..4l+3,
// so a pair's other half is in the same lane (interleaved) or R / 8 lanes away.  Many rows go 16 at a time
// (rope_rows_kernel), which is what 8192 rows of 48 heads spend 72 us in: 200 MB moved at 2.8 TB/s (the copy rate
// would allow 30 us).  No unit is saturated: 130 instructions a vector keep the issue slots 57 % busy with the 24 warps
// an SM that 80 registers leave, and what fills the rest is latency (of each instruction's result 1.7 warps, loads 1.2,
// instruction fetches 1.0, shared memory 0.8, barriers 0.5).  64 rows are one launch's latency: 4 us.
#include "kvq_append_device.cuh"

namespace kvq {
namespace {

// RN32(a c + b s): both products and the sum with their errors.
static __device__ __noinline__ float turn_exact(float a, float c, float b, float s) {
  const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p);
  const float w = __fmul_rn(b, s), we = __fmaf_rn(b, s, -w);
  const float d = __fadd_rn(p, w);
  const float v = __fsub_rn(d, p);
  const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(d, v)), __fsub_rn(w, v));
  const float rest = __fadd_rn(e, __fadd_rn(pe, we));
  // an infinite product has no error term, and a zero keeps its sign
  return fabsf(d) <= 3.4028234663852886e38f && rest != 0.f ? __fadd_rn(d, rest) : d;
}

// What turns a lane's four dims: y_j = x_j c_j + m_j s_j with m_j the other half of the pair (its sine's
// sign in s_j); dims behind R have c = 1, s = 0.
struct Turn {
  float c[4], s[4];
};
__device__ __forceinline__ Turn load_turn(const float* cs, int R, bool interleaved, int lane) {
  const int d = 4 * lane;
  Turn t;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    t.c[j] = 1.f;
    t.s[j] = 0.f;
  }
  if (d >= R) return t;
  if (interleaved) {
    const float4 v = *reinterpret_cast<const float4*>(cs + d);
    t.c[0] = t.c[1] = v.x;
    t.c[2] = t.c[3] = v.z;
    t.s[0] = -v.y;
    t.s[1] = v.y;
    t.s[2] = -v.w;
    t.s[3] = v.w;
  } else {
    const bool low = d < (R >> 1);
    const float4* p = reinterpret_cast<const float4*>(cs + 2 * (low ? d : d - (R >> 1)));
    const float4 a = p[0], b = p[1];
    const float f = low ? -1.f : 1.f;
    t.c[0] = a.x;
    t.c[1] = a.z;
    t.c[2] = b.x;
    t.c[3] = b.z;
    t.s[0] = f * a.y;
    t.s[1] = f * a.w;
    t.s[2] = f * b.y;
    t.s[3] = f * b.w;
  }
  return t;
}

// One lane's four bf16 values turned and rounded to bf16.  A product, a fused product and sum, and a bound
// on their error (2^-22 of the terms, twice what it can be): where both ends of it round to the same bf16
// value that is the exact one's; otherwise (a value in 10^4) the exact sum decides.
__device__ __forceinline__ uint2 rotate4(uint2 raw, const Turn& t, int R, bool interleaved, int lane) {
  float x[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u), __uint_as_float(raw.y << 16),
                __uint_as_float(raw.y & 0xFFFF0000u)};
  uint2 other;
  if (interleaved) {
    other = make_uint2(__byte_perm(raw.x, 0, 0x1032), __byte_perm(raw.y, 0, 0x1032));
  } else {
    const int d = 4 * lane, step = R >> 3;
    const int mate = d < R ? (d < (R >> 1) ? lane + step : lane - step) : lane;
    other = make_uint2(__shfl_sync(kFull, raw.x, mate), __shfl_sync(kFull, raw.y, mate));
  }
  const float m[4] = {__uint_as_float(other.x << 16), __uint_as_float(other.x & 0xFFFF0000u),
                      __uint_as_float(other.y << 16), __uint_as_float(other.y & 0xFFFF0000u)};
  float hi[4], lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float w = __fmul_rn(m[j], t.s[j]);
    const float y = __fmaf_rn(x[j], t.c[j], w);
    const float e = __fmul_rn(__fadd_rn(fabsf(w), fabsf(y)), 0x1p-22f);
    hi[j] = __fadd_rn(y, e);
    lo[j] = __fsub_rn(y, e);
  }
  uint2 y = make_uint2(pack_bf162(hi[0], hi[1]), pack_bf162(hi[2], hi[3]));
  if (y.x != pack_bf162(lo[0], lo[1]) || y.y != pack_bf162(lo[2], lo[3])) {
#pragma unroll
    for (int j = 0; j < 4; ++j) hi[j] = turn_exact(x[j], t.c[j], m[j], t.s[j]);
    y = make_uint2(pack_bf162(hi[0], hi[1]), pack_bf162(hi[2], hi[3]));
  }
  return 4 * lane < R ? y : raw;
}

__device__ __forceinline__ void unpack4(uint2 v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xFFFF0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}

// Row r's position in the table, or -1 (flagged by the caller).
__device__ __forceinline__ int rope_row(const RopeArgs& a, int r) {
  const int p = a.rope_pos[r];
  return p >= 0 && p < a.max_pos ? p : -1;
}

__global__ void __launch_bounds__(256) rope_append_kernel(const RopeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long vec = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int H = a.ap.c.H, per_row = a.Hq + (a.write ? 2 * H : 0);
  if (vec >= (long long)a.ap.n * per_row) return;
  const int r = int(vec / per_row), i = int(vec % per_row);
  const int rp = rope_row(a, r);
  if (rp < 0) {
    if (lane == 0) flag(a.ap.err, KVQ_DEVERR_POSITION);
    return;
  }
  const float* cs = a.table + size_t(rp) * a.R;
  if (i < a.Hq) {
    const uint2 x = *reinterpret_cast<const uint2*>(a.q + r * a.q_stride + i * kHeadDim + 4 * lane);
    *reinterpret_cast<uint2*>(a.q_out + (size_t(r) * a.Hq + i) * kHeadDim + 4 * lane) =
        rotate4(x, load_turn(cs, a.R, a.interleaved, lane), a.R, a.interleaved, lane);
    return;
  }
  const bool is_key = i < a.Hq + H;
  const int h = is_key ? i - a.Hq : i - a.Hq - H;
  uint2 v = *reinterpret_cast<const uint2*>(
      (is_key ? a.ap.k_new + r * a.k_stride : a.ap.v_new + r * a.v_stride) + h * kHeadDim + 4 * lane);
  const int b = a.ap.seq_idx[r];
  const int p = a.ap.pos[r];
  if (b < 0 || b >= a.ap.batch || p < 0 || (a.ap.mode != KVQ_APPEND_QUANT && b >= a.ap.c.window_batch)) {
    if (lane == 0) flag(a.ap.err, KVQ_DEVERR_POSITION);
    return;
  }
  if (is_key) v = rotate4(v, load_turn(cs, a.R, a.interleaved, lane), a.R, a.interleaved, lane);
  const uint16_t xb[4] = {uint16_t(v.x & 0xFFFF), uint16_t(v.x >> 16), uint16_t(v.y & 0xFFFF), uint16_t(v.y >> 16)};
  append_vector(a.ap, is_key, b, p, h, xb, lane);
}

// 2-bit caches: whole blocks, one warp per (run of rows, head, K or V).
__global__ void __launch_bounds__(kGroupWarps * 32) rope_append_group_kernel(const RopeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t img[kGroupWarps][kBlock * kHeadDim * 2 / 32];
  const int lane = threadIdx.x & 31, wslot = threadIdx.x >> 5;
  const long long vec = (long long)blockIdx.x * kGroupWarps + wslot;
  const int H = a.ap.c.H;
  if (vec >= (long long)a.ap.n * 2 * H) return;
  const int r = int(vec / (2 * H));
  const bool is_key = ((vec / H) % 2) == 0;
  const int h = int(vec % H);
  append_group(
      a.ap, r, is_key, h, img[wslot], lane, [&](int row) { return rope_row(a, row) >= 0; },
      [&](int row, float(&x)[4]) {
        uint2 v = *reinterpret_cast<const uint2*>(
            (is_key ? a.ap.k_new + row * a.k_stride : a.ap.v_new + row * a.v_stride) + h * kHeadDim + 4 * lane);
        if (is_key) {
          const Turn t = load_turn(a.table + size_t(rope_row(a, row)) * a.R, a.R, a.interleaved, lane);
          v = rotate4(v, t, a.R, a.interleaved, lane);
        }
        unpack4(v, x);
      });
}

// ---- many rows: 16 rows of the call per CTA
//
// A row at a time, a value vector's codes are 128 single bytes (or nibbles) spread over its whole
// block, and every warp waits for its own loads: 185 us for 8192 rows that take 27 us to move.
// Here (72 us) a CTA takes a window of 16 rows.  Where 16 rows of the call fill one block (a run of 16 positions
// from a multiple of 16: prompts), a warp turns and quantizes the 16 vectors of a head, puts the block
// together in shared memory and writes it as it lies, 16 bytes a lane; rows outside such runs are
// written one by one.  The window's rows of the table are staged once for all heads; queries go 8
// vectors at a time, their loads ahead of their work.
constexpr int kRows = 16;

struct RopeSmem {
  alignas(16) float cs[2 * kRows][kHeadDim];      // table rows of the window and of the run
  alignas(16) uint8_t img[8][kBlock * kHeadDim * 2];  // one block image per warp
  int seq[3 * kRows], pos[3 * kRows], rope[3 * kRows];  // rows r0 - 15 .. r0 + 32 (-1: no such row)
  int lead;           // first row of the run in this window, or -1
  unsigned single;    // rows of the window that are written one by one
};

// Codes of tokens 2t, 2t + 8, 2t + 1, 2t + 9 (lane l: dims 4l..4l+3; u: stored byte, nibble or bf16 bits)
// into the image of a key or value block.
template <int BITS, bool KEY>
__device__ __forceinline__ void put_tokens(uint8_t* img, int t, const uint32_t (&u)[4][4], int lane) {
  if constexpr (KEY) {
    const int q = lane >> 3, e = (4 * lane) & 31;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int g = 2 * t + (k >> 1), hi = k & 1, at = (4 * g + q) * 16;  // token g + 8 hi
      if constexpr (BITS == 8) {
        *reinterpret_cast<uint32_t*>(img + (2 * hi + (e >> 4)) * 512 + at + (e & 15)) =
            u[k][0] | u[k][1] << 8 | u[k][2] << 16 | u[k][3] << 24;
      } else if constexpr (BITS == 4) {
        // dims 4l..4l+3 are nibbles 2p, 2p + 4, 2p + 1, 2p + 5 (p = lane & 1) of a word shared with lane ^ 1
        const uint32_t part = (u[k][0] | u[k][1] << 16 | u[k][2] << 4 | u[k][3] << 20) << (8 * (lane & 1));
        const uint32_t word = part | __shfl_xor_sync(kFull, part, 1);
        if ((lane & 1) == 0) *reinterpret_cast<uint32_t*>(img + hi * 512 + at + (e >> 3) * 4) = word;
      } else {
        *reinterpret_cast<uint2*>(img + (4 * hi + (e >> 3)) * 512 + at + 2 * (e & 7)) =
            make_uint2(u[k][0] | u[k][1] << 16, u[k][2] | u[k][3] << 16);
      }
    }
  } else {
    const int mt = lane >> 2, hi = (lane & 3) >> 1;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint8_t* at = img + (4 * (4 * (lane & 1) + d) + t) * 16;
      if constexpr (BITS == 8) {
        *reinterpret_cast<uint32_t*>(at + (mt >> 1) * 512 + (2 * (mt & 1) + hi) * 4) =
            u[0][d] | u[1][d] << 8 | u[2][d] << 16 | u[3][d] << 24;
      } else if constexpr (BITS == 4) {
        // dims d and d + 8 (lane ^ 2) share a word: nibbles 0, 4, 1, 5 and 2, 6, 3, 7
        const uint32_t part = (u[0][d] | u[1][d] << 16 | u[2][d] << 4 | u[3][d] << 20) << (8 * hi);
        const uint32_t word = part | __shfl_xor_sync(kFull, part, 2);
        if (hi == 0) *reinterpret_cast<uint32_t*>(at + (mt >> 2) * 512 + (mt & 3) * 4) = word;
      } else {
        *reinterpret_cast<uint2*>(at + mt * 512 + 8 * hi) =
            make_uint2(u[0][d] | u[1][d] << 16, u[2][d] | u[3][d] << 16);
      }
    }
  }
}

// One full block of head h: tokens r .. r + 15 of the call, four at a time in a loop: unrolled over the 16
// tokens the kernel waited on instruction fetches (6.6 of 12 stalled warps; 209 us for 8192 rows).
template <int BITS, bool KEY>
__device__ __forceinline__ void write_block(const RopeArgs& a, RopeSmem* sm, int r, int h, uint8_t* img, int lane) {
  const CacheView& c = a.ap.c;
  const long long stride = KEY ? a.k_stride : a.v_stride;
  const uint16_t* src = (KEY ? a.ap.k_new : a.ap.v_new) + r * stride + h * kHeadDim + 4 * lane;
  auto token = [](int t, int k) { return 2 * t + (k >> 1) + 8 * (k & 1); };
  uint2 next[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) next[k] = *reinterpret_cast<const uint2*>(src + token(0, k) * stride);
  const int b = sm->seq[r - blockIdx.x * kRows + kRows - 1], p = sm->pos[r - blockIdx.x * kRows + kRows - 1];
  if (p / kBlock >= a.ap.mbps) {
    if (lane == 0) flag(a.ap.err, KVQ_DEVERR_POSITION);
    return;
  }
  const int phys = a.ap.table[size_t(b) * a.ap.mbps + p / kBlock];
  if (phys < 0 || phys >= c.num_blocks) {
    if (lane == 0) flag(a.ap.err, KVQ_DEVERR_BLOCK_ID);
    return;
  }
  float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
  if (KEY && c.factor) f = *reinterpret_cast<const float4*>(c.factor + h * kHeadDim + 4 * lane);
  float s_of = 1.f, z_of = 0.f;  // lane i < 16: token i's scale and zero point
#pragma unroll 1
  for (int t = 0; t < 4; ++t) {
    uint2 raw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      raw[k] = next[k];
      if (t < 3) next[k] = *reinterpret_cast<const uint2*>(src + token(t + 1, k) * stride);
    }
    uint32_t u[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int tok = token(t, k);
      uint2 bits = raw[k];
      if constexpr (KEY)
        bits = rotate4(bits, load_turn(sm->cs[kRows + tok], a.R, a.interleaved, lane), a.R, a.interleaved, lane);
      float x[4];
      unpack4(bits, x);
      if constexpr (BITS == 16) {
        u[k][0] = bits.x & 0xFFFFu;
        u[k][1] = bits.x >> 16;
        u[k][2] = bits.y & 0xFFFFu;
        u[k][3] = bits.y >> 16;
      } else {
        float s = 1.f, m = 0.f;
        constexpr int kBias = BITS == 8 ? 128 : 8, kTop = BITS == 8 ? 127 : 7;
        if (KEY && c.k_chan) {
          const float ff[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            u[k][j] = int(fminf(float(kTop), fmaxf(BITS == 8 ? -127.f : -8.f, round_quotient_far(x[j], ff[j])))) + kBias;
        } else {
          if (KEY && c.factor) {
            x[0] = __fdiv_rn(x[0], f.x);
            x[1] = __fdiv_rn(x[1], f.y);
            x[2] = __fdiv_rn(x[2], f.z);
            x[3] = __fdiv_rn(x[3], f.w);
          }
          if (c.asym) {
            const AsymCodes ac = quantize_asym_far(make_float4(x[0], x[1], x[2], x[3]), BITS);
#pragma unroll
            for (int j = 0; j < 4; ++j) u[k][j] = uint32_t(ac.u[j]);
            s = ac.s;
            m = ac.m;
          } else {
            int code[4];
            quantize_warp(x, BITS, code, s);
#pragma unroll
            for (int j = 0; j < 4; ++j) u[k][j] = uint32_t(code[j] + kBias);
          }
        }
        if (lane == tok) {
          s_of = s;
          z_of = m;
        }
      }
    }
    put_tokens<BITS, KEY>(img, t, u, lane);
  }
  __syncwarp();
  constexpr int kBytes = block_bytes(BITS);
  uint8_t* blk = (KEY ? c.k_codes : c.v_codes) + (size_t(h) * c.num_blocks + phys) * kBytes;
#pragma unroll
  for (int i = 0; i < kBytes / 512; ++i)
    reinterpret_cast<uint4*>(blk)[i * 32 + lane] = reinterpret_cast<const uint4*>(img)[i * 32 + lane];
  if (BITS != 16 && lane < kBlock && !(KEY && c.k_chan)) {
    float* rec = c.meta + (size_t(h) * c.num_blocks + phys) * c.meta_floats + (KEY ? 0 : c.meta_floats / 2);
    rec[lane] = s_of;
    if (c.asym) rec[kBlock + lane] = z_of;
  }
  __syncwarp();  // the image is free for the warp's next block
}

static __device__ __noinline__ void append_single(const AppendArgs& a, bool is_key, int b, int p, int h, uint2 v, int lane) {
  const uint16_t xb[4] = {uint16_t(v.x & 0xFFFF), uint16_t(v.x >> 16), uint16_t(v.y & 0xFFFF), uint16_t(v.y >> 16)};
  append_vector(a, is_key, b, p, h, xb, lane);
}

template <int KB, int VB>
__global__ void __launch_bounds__(256, 3) rope_rows_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) uint8_t raw_smem[];
  RopeSmem* sm = reinterpret_cast<RopeSmem*>(raw_smem);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.ap.c.H, n = a.ap.n, r0 = blockIdx.x * kRows, R4 = a.R / 4;
  // ---- the rows around the window, and the run in it
  if (tid < 3 * kRows) {
    const int r = r0 - (kRows - 1) + tid;
    const bool in = r >= 0 && r < n;
    sm->seq[tid] = in && a.write ? a.ap.seq_idx[r] : -1;
    sm->pos[tid] = in && a.write ? a.ap.pos[r] : -1;
    sm->rope[tid] = in ? rope_row(a, r) : -1;
  }
  __syncthreads();
  if (warp == 0) {
    // bit i: row r0 - 15 + i.  A row leads a run if 16 rows from it are one sequence's positions p, p + 1, .. with p a
    // multiple of 16, all of them with a rope position; at most one row of a window does
    auto bits = [&](int i, unsigned& first, unsigned& next, unsigned& there) {
      const bool in = i < 3 * kRows, on = in && sm->rope[i] >= 0;
      const int b = in ? sm->seq[i] : -1, p = in ? sm->pos[i] : -1;
      first = __ballot_sync(kFull, on && b >= 0 && b < a.ap.batch && p >= 0 && p % kBlock == 0);
      next = __ballot_sync(kFull, on && i + 1 < 3 * kRows && sm->rope[i + 1] >= 0 && sm->seq[i + 1] == b &&
                                      p >= 0 && sm->pos[i + 1] == p + 1);
      there = __ballot_sync(kFull, on);
    };
    unsigned first, next_lo, next_hi, there, unused[2];
    bits(lane, first, next_lo, there);
    bits(32 + lane, unused[0], next_hi, unused[1]);
    unsigned long long next = next_lo | (unsigned long long)next_hi << 32;
    next &= next >> 1;
    next &= next >> 2;
    next &= next >> 4;
    const unsigned runs = first & unsigned(next & next >> 7);  // 15 rows that the next one follows
    unsigned covered = runs | runs << 1;
    covered |= covered << 2;
    covered |= covered << 4;
    covered |= covered << 8;
    const unsigned leads = runs >> (kRows - 1) & 0xFFFFu;
    if (lane == 0) {
      sm->lead = leads ? r0 + __ffs(leads) - 1 : -1;
      // rows in no run of this window's or the one before: those are written one by one
      sm->single = a.write ? (there & ~covered) >> (kRows - 1) & 0xFFFFu : 0u;
    }
  }
  __syncthreads();
  const int lead = sm->lead;
  auto rope_of = [&](int row) {  // row 0..15 of the window, 16..31 of the run
    const int at = row < kRows ? row : (lead >= 0 ? lead - r0 + row - kRows : -1);
    return at >= 0 ? sm->rope[at + kRows - 1] : -1;
  };
  for (int i = tid; i < 2 * kRows * R4; i += 256) {
    const int row = i / R4, at = i % R4, rp = rope_of(row);
    if (rp >= 0)
      reinterpret_cast<float4*>(sm->cs[row])[at] = reinterpret_cast<const float4*>(a.table + size_t(rp) * a.R)[at];
  }
  if (tid < kRows && r0 + tid < n && rope_of(tid) < 0 && blockIdx.y == 0) flag(a.ap.err, KVQ_DEVERR_POSITION);
  __syncthreads();

  // ---- tasks: the run's blocks, the single rows' vectors, the queries 8 at a time
  const int blocks = lead >= 0 ? 2 * H : 0, singles = sm->single ? 2 * H : 0;
  const int q8 = (a.Hq + 7) / 8, queries = kRows * q8;
  const int step = 8 * gridDim.y;
  for (int task = blockIdx.y * 8 + warp; task < blocks + singles + queries; task += step) {
    if (task < blocks) {
      if (task < H) write_block<KB, true>(a, sm, lead, task, sm->img[warp], lane);
      else write_block<VB, false>(a, sm, lead, task - H, sm->img[warp], lane);
      continue;
    }
    if (task < blocks + singles) {
      const bool is_key = task - blocks < H;
      const int h = is_key ? task - blocks : task - blocks - H;
      for (unsigned left = sm->single; left; left &= left - 1) {
        const int i = __ffs(left) - 1, r = r0 + i, s = i + kRows - 1;
        const int b = sm->seq[s], p = sm->pos[s];
        if (b < 0 || b >= a.ap.batch || p < 0) {
          if (lane == 0) flag(a.ap.err, KVQ_DEVERR_POSITION);
          continue;
        }
        uint2 v = *reinterpret_cast<const uint2*>(
            (is_key ? a.ap.k_new + (long long)r * a.k_stride : a.ap.v_new + (long long)r * a.v_stride) + h * kHeadDim +
            4 * lane);
        if (is_key) v = rotate4(v, load_turn(sm->cs[i], a.R, a.interleaved, lane), a.R, a.interleaved, lane);
        append_single(a.ap, is_key, b, p, h, v, lane);
      }
      continue;
    }
    const int qt = task - blocks - singles, i = qt / q8, h0 = (qt % q8) * 8, r = r0 + i;
    if (r >= n || sm->rope[i + kRows - 1] < 0) continue;
    const uint16_t* src = a.q + (long long)r * a.q_stride + h0 * kHeadDim + 4 * lane;
    uint2 raw[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      raw[k] = h0 + k < a.Hq ? *reinterpret_cast<const uint2*>(src + k * kHeadDim) : make_uint2(0u, 0u);
    uint16_t* dst = a.q_out + ((size_t)r * a.Hq + h0) * kHeadDim + 4 * lane;
    const Turn t = load_turn(sm->cs[i], a.R, a.interleaved, lane);
#pragma unroll 1
    for (int k = 0; k < 8; k += 2) {  // a short loop; the registers rotate, so that every index is known
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint2 y = rotate4(raw[e], t, a.R, a.interleaved, lane);
        if (h0 + k + e < a.Hq) *reinterpret_cast<uint2*>(dst + (k + e) * kHeadDim) = y;
      }
#pragma unroll
      for (int e = 0; e < 6; ++e) raw[e] = raw[e + 2];
    }
  }
}

template <int KB, int VB>
cudaError_t launch_rows(const RopeArgs& a, int sms, cudaStream_t s) {
  constexpr int smem = int(sizeof(RopeSmem));
  const auto k = rope_rows_kernel<KB, VB>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int windows = (a.ap.n + kRows - 1) / kRows;
  const int tasks = (a.write ? 4 * a.ap.c.H : 0) + kRows * ((a.Hq + 7) / 8);
  // few windows: their tasks over several CTAs, up to two tasks a warp
  int y = (8 * sms + windows - 1) / windows;
  y = y > (tasks + 15) / 16 ? (tasks + 15) / 16 : y;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(windows), unsigned(y < 1 ? 1 : y));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

__global__ void __launch_bounds__(256) rope_table_kernel(const RopeFreqs f, int pairs, long long n, float* table) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  double s, c;
  sincos(double(i / pairs) * f.f[i % pairs], &s, &c);
  reinterpret_cast<float2*>(table)[i] = make_float2(float(f.amplitude * c), float(f.amplitude * s));
}

cudaError_t launch_pdl(void (*kernel)(const RopeArgs), const RopeArgs& a, long long warps, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((warps + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t s) {
  const int kb = a.ap.c.k_bits, vb = a.ap.c.v_bits;
  const bool group = a.write && kb == 2 && a.ap.mode == KVQ_APPEND_QUANT;
  // Windows of 16 rows from three waves of one-vector warps on (152 SMs x 64 warps; with the read-back, 48
  // vectors a row: 256 rows take 21 us one by one and 31 in windows, 640 33 and 31, 1024 39 and 35, 2048
  // 58 and 46; 12 vectors a row: 1024 rows 23 and 34, 2048 31 and 33): a window has more to do before its first store.
  constexpr long long kRowsVectors = 3ll * 152 * 64;
  const long long vectors = (long long)a.ap.n * (a.Hq + (a.write ? 2 * a.ap.c.H : 0));
  if (vectors >= kRowsVectors && (!a.write || (a.ap.mode == KVQ_APPEND_QUANT && !group))) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if (!a.write || (kb == 8 && vb == 8)) return launch_rows<8, 8>(a, sms, s);  // queries alone: any format
    if (kb == 4 && vb == 4) return launch_rows<4, 4>(a, sms, s);
    if (kb == 4 && vb == 8) return launch_rows<4, 8>(a, sms, s);
    if (kb == 8 && vb == 4) return launch_rows<8, 4>(a, sms, s);
    return launch_rows<16, 16>(a, sms, s);
  }
  if (!group) {
    return launch_pdl(rope_append_kernel, a, vectors, s);
  }
  if (a.Hq > 0) {
    RopeArgs q = a;
    q.write = false;
    const cudaError_t e = launch_rope_append(q, s);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(rope_append_group_kernel, a, (long long)a.ap.n * 2 * a.ap.c.H, s);
}

cudaError_t launch_rope_table(const RopeFreqs& f, int pairs, int max_pos, float* table, cudaStream_t s) {
  const long long n = (long long)max_pos * pairs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((n + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, rope_table_kernel, f, pairs, n, table);
}

}  // namespace kvq
