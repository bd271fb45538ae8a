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
// Rounding.  The two products and their sum are carried with their rounding
// errors, so y is the exact value rounded once to float32 (up to one case in
// about 2^24) and then to bf16.  That makes the stored codes those of kvq_append on the
// rotated vectors bit for bit: a plain float32 sum differs from the exact one
// in its last bit often enough to move a bf16 rounding, with it a vector's
// largest value, and with that a whole vector's codes.  It costs 14 instead of 3
// instructions per value, which the loads hide.
//
// One warp turns and writes one 128-element vector; lane l owns dims 4l..4l+3,
// so a pair's other half is in the same lane (interleaved) or R / 8 lanes away.
#include "kvq_append_device.cuh"

namespace kvq {
namespace {

// RN32(a c - b s): both products and the difference with their errors.
__device__ __forceinline__ float turn(float a, float c, float b, float s) {
  const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p);
  const float w = __fmul_rn(b, s), we = __fmaf_rn(b, s, -w);
  const float d = __fsub_rn(p, w);
  const float v = __fsub_rn(d, p);
  const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, v)), __fadd_rn(w, v));
  const float rest = __fadd_rn(e, __fsub_rn(pe, we));
  // an infinite product has no error term, and a zero keeps its sign
  return fabsf(d) <= 3.4028234663852886e38f && rest != 0.f ? __fadd_rn(d, rest) : d;
}

// One lane's four values turned by the table row cs (R / 2 pairs of cos, sin).
__device__ __forceinline__ void rotate4(float (&x)[4], const float* cs, int R, bool interleaved, int lane) {
  const int d = 4 * lane;
  if (interleaved) {
    if (d < R) {
      const float4 t = *reinterpret_cast<const float4*>(cs + d);
      const float a0 = x[0], b0 = x[1], a1 = x[2], b1 = x[3];
      x[0] = turn(a0, t.x, b0, t.y);
      x[1] = turn(a0, t.y, b0, -t.x);
      x[2] = turn(a1, t.z, b1, t.w);
      x[3] = turn(a1, t.w, b1, -t.z);
    }
    return;
  }
  const int half = R >> 1;
  const bool low = d < half;
  const int mate = d < R ? (low ? lane + (R >> 3) : lane - (R >> 3)) : lane;
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = __shfl_sync(kFull, x[j], mate);
  if (d < R) {
    const float4* t = reinterpret_cast<const float4*>(cs + 2 * (low ? d : d - half));
    const float4 t0 = t[0], t1 = t[1];
    const float c[4] = {t0.x, t0.z, t1.x, t1.z}, s[4] = {t0.y, t0.w, t1.y, t1.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = low ? turn(x[j], c[j], y[j], s[j]) : turn(y[j], s[j], x[j], -c[j]);
  }
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

__device__ __forceinline__ bool rope_row_ok(const RopeArgs& a, int r) { return rope_row(a, r) >= 0; }

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
    float x[4];
    unpack4(*reinterpret_cast<const uint2*>(a.q + r * a.q_stride + i * kHeadDim + 4 * lane), x);
    rotate4(x, cs, a.R, a.interleaved, lane);
    const uint2 y = make_uint2(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]));
    *reinterpret_cast<uint2*>(a.q_out + (size_t(r) * a.Hq + i) * kHeadDim + 4 * lane) = y;
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
  if (is_key) {
    float x[4];
    unpack4(v, x);
    rotate4(x, cs, a.R, a.interleaved, lane);
    v = make_uint2(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]));
  }
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
        unpack4(*reinterpret_cast<const uint2*>(
                    (is_key ? a.ap.k_new + row * a.k_stride : a.ap.v_new + row * a.v_stride) + h * kHeadDim + 4 * lane),
                x);
        if (!is_key) return;
        rotate4(x, a.table + size_t(rope_row(a, row)) * a.R, a.R, a.interleaved, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __bfloat162float(__float2bfloat16_rn(x[j]));
      });
}

// ---- many rows: 16 rows of the call per CTA
//
// A row at a time, a value vector's codes are 128 single bytes (or nibbles) spread over its whole
// block, and every warp waits for its own loads: 185 us for 8192 rows that take 27 us to move.
// Here a CTA takes a window of 16 rows.  Where 16 rows of the call fill one block (a run of 16 positions
// from a multiple of 16: prompts), a warp turns and quantizes the 16 vectors of a head, puts the block
// together in shared memory and writes it as it lies, 16 bytes a lane; rows outside such runs are
// written one by one.  The window's rows of the table are staged once for all heads; queries go 8
// vectors at a time, their loads ahead of their work.
constexpr int kRows = 16;

struct RopeSmem {
  alignas(16) float cs[2 * kRows][kHeadDim];      // table rows of the window and of the run
  alignas(16) uint8_t img[8][kBlock * kHeadDim * 2];  // one block image per warp
  int rp[2 * kRows];                 // rope positions (-1: none) of rows r0 .. r0 + 15, then of the run's
  int seq[3 * kRows], pos[3 * kRows];  // rows r0 - 15 .. r0 + 31 (seq -1: no such row)
  int lead;                          // first row of the run in this window, or -1
};

// Codes of 16 tokens (lane l: dims 4l..4l+3; u: stored byte, nibble or bf16 bits of token i) into the
// image of a key or value block.
template <int BITS, bool KEY>
__device__ __forceinline__ void put_block(uint8_t* img, const uint32_t (&u)[kBlock][4], int lane) {
  if constexpr (KEY) {
    const int t = lane >> 3, e = (4 * lane) & 31;
#pragma unroll
    for (int i = 0; i < kBlock; ++i) {
      const int g = i & 7, hi = i >> 3, at = (4 * g + t) * 16;
      if constexpr (BITS == 8) {
        *reinterpret_cast<uint32_t*>(img + (2 * hi + (e >> 4)) * 512 + at + (e & 15)) =
            u[i][0] | u[i][1] << 8 | u[i][2] << 16 | u[i][3] << 24;
      } else if constexpr (BITS == 4) {
        // dims 4l..4l+3 are nibbles 2q, 2q + 4, 2q + 1, 2q + 5 (q = lane & 1) of a word shared with lane ^ 1
        const uint32_t part = (u[i][0] | u[i][1] << 16 | u[i][2] << 4 | u[i][3] << 20) << (8 * (lane & 1));
        const uint32_t word = part | __shfl_xor_sync(kFull, part, 1);
        if ((lane & 1) == 0) *reinterpret_cast<uint32_t*>(img + hi * 512 + at + (e >> 3) * 4) = word;
      } else {
        *reinterpret_cast<uint2*>(img + (4 * hi + (e >> 3)) * 512 + at + 2 * (e & 7)) =
            make_uint2(u[i][0] | u[i][1] << 16, u[i][2] | u[i][3] << 16);
      }
    }
  } else {
    const int mt = lane >> 2, hi = (lane & 3) >> 1;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int g = 4 * (lane & 1) + d;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        // tokens 2t, 2t + 8, 2t + 1, 2t + 9 of this dim
        const uint32_t a = u[2 * t][d], b = u[2 * t + 8][d], c = u[2 * t + 1][d], e = u[2 * t + 9][d];
        uint8_t* at = img + (4 * g + t) * 16;
        if constexpr (BITS == 8) {
          *reinterpret_cast<uint32_t*>(at + (mt >> 1) * 512 + (2 * (mt & 1) + hi) * 4) = a | b << 8 | c << 16 | e << 24;
        } else if constexpr (BITS == 4) {
          // dims d and d + 8 (lane ^ 2) share a word: nibbles 0, 4, 1, 5 and 2, 6, 3, 7
          const uint32_t part = (a | b << 16 | c << 4 | e << 20) << (8 * hi);
          const uint32_t word = part | __shfl_xor_sync(kFull, part, 2);
          if (hi == 0) *reinterpret_cast<uint32_t*>(at + (mt >> 2) * 512 + (mt & 3) * 4) = word;
        } else {
          *reinterpret_cast<uint2*>(at + mt * 512 + 8 * hi) = make_uint2(a | b << 16, c | e << 16);
        }
      }
    }
  }
}

// One full block of head h: tokens r .. r + 15 of the call.
template <int BITS, bool KEY>
__device__ __forceinline__ void write_block(const RopeArgs& a, RopeSmem* sm, int r, int h, uint8_t* img, int lane) {
  const CacheView& c = a.ap.c;
  uint2 raw[kBlock];
  const uint16_t* src =
      (KEY ? a.ap.k_new + (long long)r * a.k_stride : a.ap.v_new + (long long)r * a.v_stride) + h * kHeadDim + 4 * lane;
  const long long stride = KEY ? a.k_stride : a.v_stride;
#pragma unroll
  for (int i = 0; i < kBlock; ++i) raw[i] = *reinterpret_cast<const uint2*>(src + i * stride);
  const int b = sm->seq[r - blockIdx.x * kRows + kRows - 1], p = sm->pos[r - blockIdx.x * kRows + kRows - 1];
  if (p + kBlock > a.ap.mbps * kBlock) {
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
  const float ff[4] = {f.x, f.y, f.z, f.w};
  uint32_t u[kBlock][4];
  float s_of = 1.f, z_of = 0.f;  // lane i < 16: token i's scale and zero point
#pragma unroll
  for (int i = 0; i < kBlock; ++i) {
    float x[4];
    unpack4(raw[i], x);
    uint2 bits = raw[i];
    if constexpr (KEY) {
      rotate4(x, sm->cs[kRows + i], a.R, a.interleaved, lane);
      bits = make_uint2(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]));
      unpack4(bits, x);
    }
    if constexpr (BITS == 16) {
      u[i][0] = bits.x & 0xFFFFu;
      u[i][1] = bits.x >> 16;
      u[i][2] = bits.y & 0xFFFFu;
      u[i][3] = bits.y >> 16;
    } else {
      int code[4];
      float s = 1.f, m = 0.f;
      constexpr int kBias = BITS == 8 ? 128 : 8, kTop = BITS == 8 ? 127 : 7;
      if (KEY && c.k_chan) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          code[j] = int(fminf(float(kTop), fmaxf(BITS == 8 ? -127.f : -8.f, round_quotient(x[j], ff[j])))) + kBias;
      } else {
        if (KEY && c.factor) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = __fdiv_rn(x[j], ff[j]);
        }
        if (c.asym) {
          quantize_asym_warp(x, BITS, code, s, m);
        } else {
          quantize_warp(x, BITS, code, s);
#pragma unroll
          for (int j = 0; j < 4; ++j) code[j] += kBias;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) u[i][j] = uint32_t(code[j]);
      if (lane == i) {
        s_of = s;
        z_of = m;
      }
    }
  }
  put_block<BITS, KEY>(img, u, lane);
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

template <int KB, int VB>
__global__ void __launch_bounds__(256, 2) rope_rows_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) uint8_t raw_smem[];
  RopeSmem* sm = reinterpret_cast<RopeSmem*>(raw_smem);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.ap.c.H, n = a.ap.n, r0 = blockIdx.x * kRows, R4 = a.R / 4;
  // ---- the rows around the window, and the run in it
  if (tid < 3 * kRows) {
    const int r = r0 - (kRows - 1) + tid;
    const bool in = a.write && r >= 0 && r < n;
    sm->seq[tid] = in ? a.ap.seq_idx[r] : -1;
    sm->pos[tid] = in ? a.ap.pos[r] : -1;
  } else if (tid >= 64 && tid < 64 + kRows) {
    const int r = r0 + tid - 64;
    sm->rp[tid - 64] = r < n ? rope_row(a, r) : -1;
  }
  if (tid == 0) sm->lead = -1;
  __syncthreads();
  if (warp == 0) {
    // row r0 + lane (lane < 16) leads a run if 16 rows from it are one sequence's positions p, p + 1, .. with
    // p a multiple of 16, all of them with a rope position; at most one row of a window does
    bool lead = lane < kRows && r0 + lane < n;
    const int s = lane < kRows ? lane + kRows - 1 : 0, b = sm->seq[s], p = sm->pos[s];
    lead = lead && b >= 0 && b < a.ap.batch && p >= 0 && p % kBlock == 0;
    for (int i = 1; i < kBlock && lead; ++i) lead = sm->seq[s + i] == b && sm->pos[s + i] == p + i;
    if (lead) {
      for (int i = 0; i < kBlock && lead; ++i) lead = rope_row(a, r0 + lane + i) >= 0;
      if (lead) sm->lead = r0 + lane;
    }
  }
  __syncthreads();
  const int lead = sm->lead;
  if (tid < kRows) sm->rp[kRows + tid] = lead >= 0 ? rope_row(a, lead + tid) : -1;
  __syncthreads();
  for (int i = tid; i < 2 * kRows * R4; i += 256) {
    const int row = i / R4, at = i % R4;
    if (sm->rp[row] >= 0)
      reinterpret_cast<float4*>(sm->cs[row])[at] =
          reinterpret_cast<const float4*>(a.table + size_t(sm->rp[row]) * a.R)[at];
  }
  if (tid < kRows && r0 + tid < n && sm->rp[tid] < 0 && blockIdx.y == 0) flag(a.ap.err, KVQ_DEVERR_POSITION);
  __syncthreads();

  // ---- tasks: the run's blocks, the single rows' vectors, the queries 8 at a time
  const int blocks = lead >= 0 ? 2 * H : 0, singles = a.write ? 2 * H : 0;
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
      for (int i = 0; i < kRows; ++i) {
        const int r = r0 + i, s = i + kRows - 1;
        if (r >= n || sm->rp[i] < 0) continue;
        const int b = sm->seq[s], p = sm->pos[s];
        if (b < 0 || b >= a.ap.batch || p < 0) {
          if (lane == 0) flag(a.ap.err, KVQ_DEVERR_POSITION);
          continue;
        }
        // part of a full run, led by row r - p % 16 of this window or the one before?  Its rows are in view.
        const int j = p % kBlock;
        bool run = s - j >= 0;
        if (run) {
          const int at = min(lane, kBlock - 1), k = s - j + at;
          run = __all_sync(kFull, sm->seq[k] == b && sm->pos[k] == p - j + at && rope_row_ok(a, r - j + at));
        }
        if (run) continue;
        uint2 v = *reinterpret_cast<const uint2*>(
            (is_key ? a.ap.k_new + (long long)r * a.k_stride : a.ap.v_new + (long long)r * a.v_stride) + h * kHeadDim +
            4 * lane);
        if (is_key) {
          float x[4];
          unpack4(v, x);
          rotate4(x, sm->cs[i], a.R, a.interleaved, lane);
          v = make_uint2(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]));
        }
        const uint16_t xb[4] = {uint16_t(v.x & 0xFFFF), uint16_t(v.x >> 16), uint16_t(v.y & 0xFFFF),
                                uint16_t(v.y >> 16)};
        append_vector(a.ap, is_key, b, p, h, xb, lane);
      }
      continue;
    }
    const int t = task - blocks - singles, i = t / q8, h0 = (t % q8) * 8, r = r0 + i;
    if (r >= n || sm->rp[i] < 0) continue;
    const uint16_t* src = a.q + (long long)r * a.q_stride + h0 * kHeadDim + 4 * lane;
    uint2 raw[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (h0 + k < a.Hq) raw[k] = *reinterpret_cast<const uint2*>(src + k * kHeadDim);
    uint16_t* dst = a.q_out + ((size_t)r * a.Hq + h0) * kHeadDim + 4 * lane;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (h0 + k >= a.Hq) break;
      float x[4];
      unpack4(raw[k], x);
      rotate4(x, sm->cs[i], a.R, a.interleaved, lane);
      *reinterpret_cast<uint2*>(dst + k * kHeadDim) = make_uint2(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]));
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
  int y = (4 * sms + windows - 1) / windows;
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
  if ((e = cudaLaunchKernelEx(&cfg, k, a)) != cudaSuccess) return e;
  return cudaGetLastError();
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t s) {
  const int kb = a.ap.c.k_bits, vb = a.ap.c.v_bits;
  const bool group = a.write && kb == 2 && a.ap.mode == KVQ_APPEND_QUANT;
  // Windows of 16 rows from kRowsMin rows on; fewer rows are one wave of single-vector warps and sooner done.
  constexpr int kRowsMin = 256;
  if (a.ap.n >= kRowsMin && (!a.write || (a.ap.mode == KVQ_APPEND_QUANT && !group))) {
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
    const long long per_row = a.Hq + (a.write ? 2 * a.ap.c.H : 0);
    return launch_pdl(rope_append_kernel, a, a.ap.n * per_row, s);
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
  rope_table_kernel<<<unsigned((n + 255) / 256), 256, 0, s>>>(f, pairs, n, table);
  return cudaGetLastError();
}

}  // namespace kvq
