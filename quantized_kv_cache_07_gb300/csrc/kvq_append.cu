// Quantize-on-write (kvq_append) and read-back (kvq_dequant) kernels.
//
// Quantizer: "KV Cache Quantization and Per-Token Scale Placement", sections
// "Per-token scales and where they can live" (one scale per token per head,
// computed at write time, stored alongside the codes) and "The axis choice is a
// kernel decision" (listing: amax, zero vector -> scale 1, scale = amax/qmax,
// clamp(round(x/scale))); "KV Cache Quantization Reduces Cache Bytes with
// Separate Accuracy and Kernel Costs", section "Quantization needs a scale
// convention" (q = clamp(round(x/s)), x_hat = q*s).  Asymmetric format: "KV
// Cache Quantization Perturbs Attention Through Stored Keys and Values",
// section "Quantization granularity defines which values share a scale" (a
// scale and a zero point per group; here per token per head).
//
// 2-bit codes share one scale (and zero point) per 16-token block: "KV Cache
// Quantization and Per-Token Scale Placement", section "Per-token scales and
// where they can live" (at 2 bits, schemes group several tokens under one
// scale).  A block is quantized as one vector of up to 16 x 128 values.
//
// One warp quantizes one 128-element vector (or one 2-bit token group); lane l
// owns dims 4l..4l+3.
#include "kvq_append_device.cuh"

namespace kvq {
namespace {

__global__ void __launch_bounds__(256) append_kernel(AppendArgs a) {
  // Programmatic dependent launch: wait for the previous kernel on the stream
  // (its writes visible) before touching memory; let the next one launch early.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long vec = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int H = a.c.H;
  if (vec >= (long long)a.n * 2 * H) return;
  const int r = int(vec / (2 * H));
  const int kv = int((vec / H) % 2);
  const int h = int(vec % H);
  const bool is_key = kv == 0;
  // the new vector does not depend on the destination: load it with the indices
  const uint16_t* src = (is_key ? a.k_new : a.v_new) + (size_t(r) * H + h) * kHeadDim + 4 * lane;
  const uint2 v_new = *reinterpret_cast<const uint2*>(src);
  const int b = a.seq_idx[r];
  const int p = a.pos[r];
  if (b < 0 || b >= a.batch || p < 0 ||
      (a.mode != KVQ_APPEND_QUANT && b >= a.c.window_batch)) {
    if (lane == 0) flag(a.err, KVQ_DEVERR_POSITION);
    return;
  }
  uint16_t xb[4];
  {
    const uint2 v = v_new;
    xb[0] = uint16_t(v.x & 0xFFFF);
    xb[1] = uint16_t(v.x >> 16);
    xb[2] = uint16_t(v.y & 0xFFFF);
    xb[3] = uint16_t(v.y >> 16);
  }
  append_vector(a, is_key, b, p, h, xb, lane);
}

__global__ void __launch_bounds__(kGroupWarps * 32) append_group_kernel(AppendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t img[kGroupWarps][kBlock * kHeadDim * 2 / 32];  // one 512-byte block per warp
  const int lane = threadIdx.x & 31, wslot = threadIdx.x >> 5;
  const long long vec = (long long)blockIdx.x * kGroupWarps + wslot;
  const int H = a.c.H;
  if (vec >= (long long)a.n * 2 * H) return;
  const int r = int(vec / (2 * H));
  const bool is_key = ((vec / H) % 2) == 0;
  const int h = int(vec % H);
  const uint16_t* src = is_key ? a.k_new : a.v_new;
  append_group(
      a, r, is_key, h, img[wslot], lane, [](int) { return true; },
      [&](int row, float(&x)[4]) {
        const uint2 v = *reinterpret_cast<const uint2*>(src + (size_t(row) * H + h) * kHeadDim + 4 * lane);
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
      });
}

__global__ void __launch_bounds__(256) dequant_kernel(DequantArgs a) {
  const int lane = threadIdx.x & 31;
  const long long vec = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int H = a.c.H;
  if (vec >= (long long)a.n * 2 * H) return;
  const int r = int(vec / (2 * H));
  const bool is_key = ((vec / H) % 2) == 0;
  const int h = int(vec % H);
  const int slot = a.slots[r];
  const int phys = slot / kBlock, tok = slot % kBlock;
  float* out = (is_key ? a.k_out : a.v_out) + (size_t(r) * H + h) * kHeadDim + 4 * lane;
  if (slot < 0 || phys >= a.c.num_blocks) {
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = 0.0f;
    return;
  }
  const int bits = is_key ? a.c.k_bits : a.c.v_bits;
  const uint8_t* blk = (is_key ? a.c.k_codes : a.c.v_codes) + (size_t(h) * a.c.num_blocks + phys) * block_bytes(bits);
  float s = 1.0f, m = 0.0f;
  const bool asym = a.c.asym != 0;
  const bool chan = is_key && a.c.k_chan;  // per-channel key scale c_j instead of a per-token one
  if (bits == 2) {
    const float* rec = a.c.meta + (size_t(h) * a.c.num_blocks + phys) * a.c.meta_floats;
    s = rec[is_key ? 0 : 2];
    m = rec[is_key ? 1 : 3];
  } else if (bits != 16 && !chan) {
    const float* rec = a.c.meta + (size_t(h) * a.c.num_blocks + phys) * a.c.meta_floats;
    const int off = is_key ? 0 : a.c.meta_floats / 2;
    s = rec[off + tok];
    if (asym) m = rec[off + kBlock + tok];
  }
  const int bias = asym ? 0 : (bits == 8 ? 128 : (bits == 4 ? 8 : 2));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int d = 4 * lane + j;
    const Loc L = is_key ? key_loc(bits, tok, d) : value_loc(bits, tok, d);
    float v;
    if (bits == 16) {
      v = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(blk + L.byte));
    } else {
      const int raw = bits == 8 ? int(blk[L.byte]) : int((blk[L.byte] >> L.shift) & (bits == 4 ? 0xF : 0x3));
      const float sd = chan ? a.c.factor[h * kHeadDim + d] : s;
      v = asym ? __fmaf_rn(float(raw), s, m) : __fmul_rn(float(raw - bias), sd);
    }
    out[j] = v;
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  const long long vecs = (long long)a.n * 2 * a.c.H;
  if (vecs == 0) return cudaSuccess;
  const bool group = a.c.k_bits == 2 && a.mode == KVQ_APPEND_QUANT;
  const int warps = group ? kGroupWarps : 8;
  const long long grid = (vecs + warps - 1) / warps;
  // launched with programmatic stream serialisation, so the launch overlaps the
  // tail of the previous kernel (the kernel waits for it before reading memory)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = group ? cudaLaunchKernelEx(&cfg, append_group_kernel, a) : cudaLaunchKernelEx(&cfg, append_kernel, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_dequant(const DequantArgs& a, cudaStream_t s) {
  const long long vecs = (long long)a.n * 2 * a.c.H;
  if (vecs == 0) return cudaSuccess;
  const int warps = 8;
  const long long grid = (vecs + warps - 1) / warps;
  dequant_kernel<<<unsigned(grid), warps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
