// Eviction by accumulated attention weight (kvq_evict): every (sequence, KV
// head) keeps its heaviest tokens, in place.
//
// Attention does not depend on the order of the cached tokens (positions are in
// the keys), so the kept ones need not be packed in order: of the K slots that
// remain, those whose token goes ("holes") are filled with the kept tokens from
// behind slot K, the i-th hole with the i-th of them.  Sources lie at or behind
// K, destinations below it, so all moves are independent of each other, nothing
// is staged, and only about keep * (1 - keep / len) of the kept tokens move.
//
// Two launches.
//   select: one CTA per unit finds the K-th largest sum by radix selection on the
//     sums' order-preserving bits (8 bits a pass), then walks the slots in order with
//     block scans for the ranks of holes and kept tail tokens and writes the source
//     of every slot.  Ties go to the lowest slot: the result is one and the same
//     whatever the scheduling.
//   move: one warp per 16-token block with holes copies codes and scales.  A key
//     token is 16-byte pieces of the fragment-native block; a value token is one
//     field (byte, nibbles or half) of every word of four lanes' pieces, merged
//     into the destination's words, which only this warp writes.
#include "kvq_decode_impl.cuh"

namespace kvq {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kWin = 16384;  // holes matched per walk (64 KB of slots); more take another walk

// What one sequence keeps: of Lq stored tokens (and the ring's), n go.
struct EvictLen {
  int L, Lq, n;
};

__device__ __forceinline__ EvictLen evict_len(const EvictArgs& a, int b, bool& bad) {
  EvictLen e;
  const int W = a.c.window;
  const long long room = min((long long)a.mbps * kBlock + W, (long long)a.stride);
  e.L = a.seq_lens[b];
  int keep = a.keep[b];
  if (e.L < 0 || e.L > room || keep < 0) {
    bad = true;
    e.L = e.L < 0 ? 0 : int(min((long long)e.L, room));
    keep = max(keep, 0);
  }
  e.Lq = max(e.L - W, 0);
  e.n = min(max(e.L - keep, 0), e.Lq);
  if (W > 0) e.n -= e.n % W;  // ring tokens keep their slots: position mod W does not change
  return e;
}

// Order-preserving bits of a sum: NaN lowest, both zeros equal.
__device__ __forceinline__ uint32_t order_bits(float m) {
  if (m != m) return 0u;
  const uint32_t u = m == 0.f ? 0u : __float_as_uint(m);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct RowKeys {
  const float* mass;
  const int* pos;  // or null: the slot
  int first, recent_from;
  __device__ __forceinline__ uint32_t operator()(int s) const {
    const int p = pos ? pos[s] : s;
    return s < first || p >= recent_from ? 0xFFFFFFFFu : order_bits(mass[s]);
  }
};

// Exclusive scan of v over the CTA and its total; two barriers.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sum, uint32_t& total, int warp, int lane) {
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t n = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += n;
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) warp_sum[warp] = s;
  __syncthreads();
  uint32_t w = lane < kSelWarps ? warp_sum[lane] : 0u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t n = __shfl_up_sync(kFull, w, o);
    if (lane >= o) w += n;
  }
  total = __shfl_sync(kFull, w, kSelWarps - 1);
  const uint32_t before = __shfl_sync(kFull, w, max(warp - 1, 0));
  return s - v + (warp > 0 ? before : 0u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t sm[];
  uint32_t* hist = sm;                   // [kSelWarps][256]
  uint32_t* warp_sum = hist + kSelWarps * 256;  // [32]
  uint32_t* pick = warp_sum + 32;        // [2]: digit, rank within it
  int* list = reinterpret_cast<int*>(pick + 2);  // [kWin]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.c.H, b = blockIdx.x / H, h = blockIdx.x % H;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  bool bad = false;
  const EvictLen e = evict_len(a, b, bad);
  const int K = e.Lq - e.n, new_len = e.L - e.n;
  if (h == 0 && tid == 0) {
    a.new_lens[b] = new_len;
    if (bad) flag(a.err, KVQ_DEVERR_SEQ_LEN);
  }
  const size_t row = size_t(blockIdx.x) * a.stride;
  int* source = a.source + row;
  const int next = a.next_pos ? a.next_pos[b] : e.L;
  const long long from = (long long)next - a.protect_recent;
  const RowKeys key{a.mass + row, a.token_pos ? a.token_pos + row : nullptr, a.protect_first,
                    int(max(from, -2147483647ll))};
  if (e.n > 0 && K > 0) {
    // ---- the K-th largest key: digits from the top, `need` keys of the prefix wanted
    uint32_t prefix = 0u, need = uint32_t(K);
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < kSelWarps * 256; i += kSelThreads) hist[i] = 0u;
      __syncthreads();
      for (int s = tid; s < e.Lq; s += kSelThreads) {
        const uint32_t k = key(s);
        if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[warp * 256 + ((k >> shift) & 255u)], 1u);
      }
      __syncthreads();
      if (tid < 256) {
        uint32_t c = 0u;
        for (int w = 0; w < kSelWarps; ++w) c += hist[w * 256 + tid];
        hist[tid] = c;  // only this thread reads hist[w * 256 + tid]
      }
      __syncthreads();
      if (warp == 0) {  // lane l: digits 255 - 8l .. 248 - 8l, from the top
        uint32_t c = 0u;
        for (int i = 0; i < 8; ++i) c += hist[255 - 8 * lane - i];
        uint32_t s = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t n = __shfl_up_sync(kFull, s, o);
          if (lane >= o) s += n;
        }
        if (s >= need && s - c < need) {  // exactly one lane
          uint32_t above = s - c;
          for (int i = 0; i < 8; ++i) {
            const uint32_t d = hist[255 - 8 * lane - i];
            if (above + d >= need) {
              pick[0] = 255 - 8 * lane - i;
              pick[1] = need - above;
              break;
            }
            above += d;
          }
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | pick[0];
      need = pick[1];
      __syncthreads();
    }
    // ---- match holes and kept tail tokens by rank: kWin ranks a walk
    uint32_t moves = 0u, w0 = 0u;
    do {
      uint32_t ties = 0u, holes = 0u, tails = 0u;
      for (int base = 0; base < e.Lq; base += kSelThreads) {
        const int s = base + tid;
        const uint32_t k = s < e.Lq ? key(s) : 0u;
        const bool tie = s < e.Lq && k == prefix;
        // ranks of ties first: of equal sums the lowest slots stay
        uint32_t total;
        const uint32_t tr = block_scan(tie ? 1u : 0u, warp_sum, total, warp, lane) + ties;
        ties += total;
        const bool kept = s < e.Lq && (k > prefix || (tie && tr < need));
        const bool hole = s < K && !kept, tail = s >= K && kept;
        const uint32_t r = block_scan((hole ? 1u : 0u) | (tail ? 0x10000u : 0u), warp_sum, total, warp, lane);
        const uint32_t hr = holes + (r & 0xFFFFu), tl = tails + (r >> 16);
        holes += total & 0xFFFFu;
        tails += total >> 16;
        if (hole && hr >= w0 && hr - w0 < kWin) list[hr - w0] = s;
        if (s < K && kept) source[s] = s;
        // a chunk may hold the last holes and the first tail tokens: the list is complete behind the barrier
        __syncthreads();
        if (tail && tl >= w0 && tl - w0 < kWin) source[list[tl - w0]] = s;
      }
      moves = holes;
      w0 += kWin;
      __syncthreads();
    } while (w0 < moves);
  } else {
    for (int s = tid; s < K; s += kSelThreads) source[s] = s;
  }
  __syncthreads();
  // ---- sums and positions follow their tokens (in place where out is in: sources are read before the
  // ring's entries move onto them)
  for (int s = tid; s < K; s += kSelThreads) {
    const int f = source[s];
    if (a.mass_out && (f != s || a.mass_out != a.mass)) a.mass_out[row + s] = a.mass[row + f];
    if (a.pos_out && (f != s || a.pos_out != a.token_pos)) a.pos_out[row + s] = a.token_pos ? a.token_pos[row + f] : f;
  }
  __syncthreads();
  for (int s = K + tid; s < new_len; s += kSelThreads) {  // the ring's tokens
    const int f = s + e.n;
    source[s] = f;
    if (a.mass_out) a.mass_out[row + s] = a.mass[row + f];
    if (a.pos_out) a.pos_out[row + s] = a.token_pos ? a.token_pos[row + f] : f;
  }
}

// Field of token i in the words of a value piece (see value_loc): i = 2t + (j >> 1) + 8 (j & 1).
__device__ __forceinline__ int value_j(int i) { return 2 * (i & 1) + (i >> 3); }

template <int VB>
__device__ __forceinline__ void move_field(uint4& d, const uint4& s, int jd, int js) {
  uint32_t dw[4] = {d.x, d.y, d.z, d.w};
  const uint32_t sw[4] = {s.x, s.y, s.z, s.w};
  if constexpr (VB == 16) {  // words (j >> 1) and 2 + (j >> 1), half j & 1
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((i & 1) == (jd >> 1)) {
        const uint32_t v = ((js >> 1) ? sw[i | 1] : sw[i & 2]) >> (16 * (js & 1)) & 0xFFFFu;
        dw[i] = (dw[i] & ~(0xFFFFu << (16 * (jd & 1)))) | (v << (16 * (jd & 1)));
      }
  } else {
    const uint32_t m = VB == 8 ? 0xFFu : 0xF0Fu;
    const int shd = VB == 8 ? 8 * jd : 4 * (jd >> 1) + 16 * (jd & 1);
    const int shs = VB == 8 ? 8 * js : 4 * (js >> 1) + 16 * (js & 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[i] = (dw[i] & ~(m << shd)) | (((sw[i] >> shs) & m) << shd);
  }
  d = make_uint4(dw[0], dw[1], dw[2], dw[3]);
}

template <int KB, int VB>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int H = a.c.H;
  const long long total = (long long)a.B * H * a.mbps;
  const long long step = (long long)gridDim.x * (blockDim.x >> 5);
  for (long long i = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < total; i += step) {
    const int u = int(i / a.mbps), blk = int(i % a.mbps), b = u / H, h = u % H;
    bool bad = false;
    const EvictLen e = evict_len(a, b, bad);
    const int K = e.Lq - e.n;
    if (e.n == 0 || blk * kBlock >= K) continue;
    const int slot = blk * kBlock + lane;
    int src = slot;
    if (lane < kBlock && slot < K) src = a.source[size_t(u) * a.stride + slot];
    bool hole = src != slot;
    if (!__any_sync(kFull, hole)) continue;
    const int* table = a.table + size_t(b) * a.mbps;
    const int dphys = table[blk];
    int sphys = hole ? table[src / kBlock] : 0;
    const bool ok = dphys >= 0 && dphys < a.c.num_blocks;
    if ((hole && (sphys < 0 || sphys >= a.c.num_blocks)) || !ok) {
      flag(a.err, KVQ_DEVERR_BLOCK_ID);
      hole = false;
    }
    const uint32_t holes = __ballot_sync(kFull, hole);
    const int stok = src % kBlock;
    const size_t hb = size_t(h) * a.c.num_blocks;
    // keys: token g + 8 hi owns the pieces of lanes 4g..4g+3 in the chunks of its half
    constexpr int kPer = KB / 4;  // 512-byte chunks per half
    uint8_t* kd = a.c.k_codes + (hb + (ok ? dphys : 0)) * block_bytes(KB);
#pragma unroll
    for (int c = 0; c < 2 * kPer; ++c) {
      const int tok = g + 8 * (c / kPer);
      const int sp = __shfl_sync(kFull, sphys, tok), st = __shfl_sync(kFull, stok, tok);
      if (holes >> tok & 1u) {
        const uint8_t* ks = a.c.k_codes + (hb + sp) * block_bytes(KB);
        reinterpret_cast<uint4*>(kd)[c * 32 + lane] =
            reinterpret_cast<const uint4*>(ks)[((st >> 3) * kPer + c % kPer) * 32 + 4 * (st & 7) + t];
      }
    }
    // values: lane t's pieces hold tokens 2t, 2t + 8, 2t + 1, 2t + 9
    uint8_t* vd = a.c.v_codes + (hb + (ok ? dphys : 0)) * block_bytes(VB);
    int sp[4], st[4];
    bool mine = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int tok = 2 * t + (j >> 1) + 8 * (j & 1);
      sp[j] = __shfl_sync(kFull, sphys, tok);
      st[j] = __shfl_sync(kFull, stok, tok);
      if (!(holes >> tok & 1u)) sp[j] = -1;
      mine = mine || sp[j] >= 0;
    }
    if (mine) {
#pragma unroll
      for (int c = 0; c < VB / 2; ++c) {
        uint4* at = reinterpret_cast<uint4*>(vd) + c * 32 + lane;
        uint4 d = *at;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (sp[j] < 0) continue;
          const uint8_t* vs = a.c.v_codes + (hb + sp[j]) * block_bytes(VB);
          move_field<VB>(d, reinterpret_cast<const uint4*>(vs)[c * 32 + 4 * g + ((st[j] & 7) >> 1)], j, value_j(st[j]));
        }
        *at = d;
      }
    }
    // scales (and zero points): token lane's entries of the record
    if (KB != 16 && hole) {
      const float* rs = a.c.meta + (hb + sphys) * a.c.meta_floats + stok;
      float* rd = a.c.meta + (hb + dphys) * a.c.meta_floats + lane;
      for (int f = 0; f < a.c.meta_floats; f += kBlock) rd[f] = rs[f];
    }
  }
}

cudaLaunchConfig_t pdl_config(int grid, int threads, int smem, cudaStream_t s, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int KB, int VB>
cudaError_t launch_move(const EvictArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const long long ctas = ((long long)a.B * a.c.H * a.mbps + 7) / 8;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(int(ctas < 8ll * sms ? ctas : 8ll * sms), 256, 0, s, attr);
  if ((e = cudaLaunchKernelEx(&cfg, evict_move_kernel<KB, VB>, a)) != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  constexpr int smem = (kSelWarps * 256 + 34 + kWin) * 4;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(a.B * a.c.H, kSelThreads, smem, s, attr);
  if ((e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a)) != cudaSuccess) return e;
  const int kb = a.c.k_bits, vb = a.c.v_bits;
  if (kb == 8 && vb == 8) return launch_move<8, 8>(a, s);
  if (kb == 4 && vb == 4) return launch_move<4, 4>(a, s);
  if (kb == 4 && vb == 8) return launch_move<4, 8>(a, s);
  if (kb == 8 && vb == 4) return launch_move<8, 4>(a, s);
  if (kb == 16 && vb == 16) return launch_move<16, 16>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
