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
  const bool group = a.write && a.ap.c.k_bits == 2 && a.ap.mode == KVQ_APPEND_QUANT;
  if (!group) {
    const long long per_row = a.Hq + (a.write ? 2 * a.ap.c.H : 0);
    return launch_pdl(rope_append_kernel, a, a.ap.n * per_row, s);
  }
  if (a.Hq > 0) {
    RopeArgs q = a;
    q.write = false;
    const cudaError_t e = launch_pdl(rope_append_kernel, q, (long long)a.ap.n * a.Hq, s);
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
