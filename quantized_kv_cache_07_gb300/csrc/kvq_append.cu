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

// Dims 4 lane..4 lane + 3 of one slot's key or value; zeros where there is no such slot.
__device__ __forceinline__ float4 dequant_load(const DequantArgs& a, int slot, bool is_key, int h, int lane) {
  const int phys = slot / kBlock, tok = slot % kBlock;
  if (slot < 0 || phys >= a.c.num_blocks) return make_float4(0.f, 0.f, 0.f, 0.f);
  float o[4];
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
    o[j] = v;
  }
  return make_float4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void dequant_store(const DequantArgs& a, int r, bool is_key, int h, int lane, float4 v) {
  float* out = (is_key ? a.k_out : a.v_out) + (size_t(r) * a.c.H + h) * kHeadDim + 4 * lane;
  if (a.wide) {
    *reinterpret_cast<float4*>(out) = v;
  } else {
    out[0] = v.x;
    out[1] = v.y;
    out[2] = v.z;
    out[3] = v.w;
  }
}

__global__ void __launch_bounds__(256) dequant_kernel(const DequantArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long vec = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int H = a.c.H;
  if (vec >= (long long)a.n * 2 * H) return;
  const int r = int(vec / (2 * H));
  const bool is_key = ((vec / H) % 2) == 0;
  const int h = int(vec % H);
  dequant_store(a, r, is_key, h, lane, dequant_load(a, a.slots[r], is_key, h, lane));
}

// Many slots: 16 rows of the call per warp and (head, K or V).  Rows whose slots follow each other in a block are
// taken together, by the warp of the 16 that the first of them lies in: the block is read as it lies, 16
// bytes a lane, into shared memory and taken apart there; a value token on its own is 128 single bytes of its
// block.  (One row after another for what is not a whole block: 17 us for 1337 slots of 8 sequences.)
constexpr int kDqWarps = 8;

template <int BITS, bool KEY>
__device__ __forceinline__ int code_at(const uint8_t* img, int tok, int lane, int j) {
  const Loc L = KEY ? key_loc(BITS, tok, 4 * lane + j) : value_loc(BITS, tok, 4 * lane + j);
  if constexpr (BITS == 16) return *reinterpret_cast<const uint16_t*>(img + L.byte);
  return BITS == 8 ? img[L.byte] : (img[L.byte] >> L.shift) & 0xF;
}

// Rows r .. r + count - 1 of the call: tokens tok0 .. of one block.
template <int BITS, bool KEY>
__device__ __forceinline__ void dequant_block(const DequantArgs& a, int r, int slot, int count, int h, uint8_t* img,
                                              int lane) {
  const CacheView& c = a.c;
  const size_t hb = size_t(h) * c.num_blocks + slot / kBlock;
  const int tok0 = slot % kBlock;
  const uint4* blk = reinterpret_cast<const uint4*>((KEY ? c.k_codes : c.v_codes) + hb * block_bytes(BITS));
#pragma unroll
  for (int i = 0; i < BITS / 2; ++i) reinterpret_cast<uint4*>(img)[i * 32 + lane] = blk[i * 32 + lane];
  float s_of = 1.f, z_of = 0.f;  // lane i: token i's scale and zero point
  const bool chan = KEY && c.k_chan;
  if (BITS != 16 && !chan && lane < kBlock) {
    const float* rec = c.meta + hb * c.meta_floats + (KEY ? 0 : c.meta_floats / 2);
    s_of = rec[lane];
    if (c.asym) z_of = rec[kBlock + lane];
  }
  float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
  if (chan) f = *reinterpret_cast<const float4*>(c.factor + h * kHeadDim + 4 * lane);
  __syncwarp();
  const int bias = c.asym ? 0 : (BITS == 8 ? 128 : 8);
#pragma unroll 4
  for (int i = 0; i < count; ++i) {
    const float s = __shfl_sync(kFull, s_of, tok0 + i), z = __shfl_sync(kFull, z_of, tok0 + i);
    const float ff[4] = {f.x, f.y, f.z, f.w};
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int raw = code_at<BITS, KEY>(img, tok0 + i, lane, j);
      if constexpr (BITS == 16) v[j] = bf16_bits_to_f32(uint16_t(raw));
      else v[j] = c.asym ? __fmaf_rn(float(raw), s, z) : __fmul_rn(float(raw - bias), chan ? ff[j] : s);
    }
    dequant_store(a, r + i, KEY, h, lane, make_float4(v[0], v[1], v[2], v[3]));
  }
  __syncwarp();
}

template <int KB, int VB>
__global__ void __launch_bounds__(kDqWarps * 32) dequant_rows_kernel(const DequantArgs a) {
  __shared__ __align__(16) uint8_t img[kDqWarps][kBlock * kHeadDim * 2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = a.c.H;
  const long long task = (long long)blockIdx.x * kDqWarps + warp;
  const long long windows = (a.n + kBlock - 1) / kBlock;
  if (task >= windows * 2 * H) return;
  const int r0 = int(task / (2 * H)) * kBlock, kv = int(task % (2 * H));
  const bool is_key = kv < H;
  const int h = is_key ? kv : kv - H;
  // rows r0 - 1 .. r0 + 30, one a lane, -1 for a row or slot that is not there
  const long long row = (long long)r0 - 1 + lane;
  int slot = row >= 0 && row < a.n ? a.slots[row] : -1;
  if (slot < 0 || slot / kBlock >= a.c.num_blocks) slot = -1;
  const int before = __shfl_up_sync(kFull, slot, 1);
  const bool follows = lane > 0 && slot >= 0 && before >= 0 && slot == before + 1 && slot % kBlock != 0;
  // bit i: row r0 + i
  const uint32_t goes_on = __ballot_sync(kFull, follows) >> 1;
  const uint32_t none = __ballot_sync(kFull, slot < 0 && row < a.n) >> 1;
  uint32_t starts = ~goes_on & ~none & 0xFFFFu;
  if (a.n - r0 < kBlock) starts &= (1u << (a.n - r0)) - 1u;
#pragma unroll 1
  while (starts) {
    const int l = __ffs(starts) - 1;
    starts &= starts - 1;
    const int first = __shfl_sync(kFull, slot, l + 1);
    const int count = __ffs(~(goes_on >> l >> 1));  // the rows behind it that go on, and itself
    if (is_key) dequant_block<KB, true>(a, r0 + l, first, count, h, img[warp], lane);
    else dequant_block<VB, false>(a, r0 + l, first, count, h, img[warp], lane);
  }
  for (uint32_t z = none & 0xFFFFu; z; z &= z - 1) {
    const int r = r0 + __ffs(z) - 1;
    if (r < a.n) dequant_store(a, r, is_key, h, lane, make_float4(0.f, 0.f, 0.f, 0.f));
  }
}

}  // namespace

// Launched with programmatic stream serialisation, so the launch overlaps the tail of the
// previous kernel (the kernels wait for it before reading memory).
template <class Kernel, class Args>
static cudaError_t launch_pdl(Kernel kernel, const Args& a, long long grid, int threads, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  const long long vecs = (long long)a.n * 2 * a.c.H;
  if (vecs == 0) return cudaSuccess;
  const bool group = a.c.k_bits == 2 && a.mode == KVQ_APPEND_QUANT;
  const int warps = group ? kGroupWarps : 8;
  const long long grid = (vecs + warps - 1) / warps;
  return group ? launch_pdl(append_group_kernel, a, grid, warps * 32, s) : launch_pdl(append_kernel, a, grid, warps * 32, s);
}

cudaError_t launch_dequant(const DequantArgs& a, cudaStream_t s) {
  const long long vecs = (long long)a.n * 2 * a.c.H;
  if (vecs == 0) return cudaSuccess;
  // 16 slots a warp from a wave of one-vector warps on (152 SMs x 64 warps; behind the rotary write, 16
  // vectors a slot: 384 slots take 30 us one by one and 33 so, 640 33 and 31, 2048 48 and 46)
  if (vecs >= 152 * 64 && a.c.k_bits != 2) {
    const long long tasks = (long long)((a.n + kBlock - 1) / kBlock) * 2 * a.c.H;
    const long long grid = (tasks + kDqWarps - 1) / kDqWarps;
    const int kb = a.c.k_bits, vb = a.c.v_bits, threads = kDqWarps * 32;
    if (kb == 8 && vb == 8) return launch_pdl(dequant_rows_kernel<8, 8>, a, grid, threads, s);
    if (kb == 4 && vb == 4) return launch_pdl(dequant_rows_kernel<4, 4>, a, grid, threads, s);
    if (kb == 4) return launch_pdl(dequant_rows_kernel<4, 8>, a, grid, threads, s);
    if (kb == 8) return launch_pdl(dequant_rows_kernel<8, 4>, a, grid, threads, s);
    return launch_pdl(dequant_rows_kernel<16, 16>, a, grid, threads, s);
  }
  return launch_pdl(dequant_kernel, a, (vecs + 7) / 8, 256, s);
}

}  // namespace kvq
