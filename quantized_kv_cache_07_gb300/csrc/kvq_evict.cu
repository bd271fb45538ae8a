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
//   select: a cluster of 1 to 8 CTAs per unit, each with a run of its slots, finds the K-th largest sum by radix
//     selection on the sums' order-preserving bits (11 bits a pass, up to three; the sums are
//     read once, their keys stay in shared memory), then ranks holes and kept tail
//     tokens by warp runs and ballots and matches them through lists in the cluster's shared
//     memory.  Ties go to the lowest slot: the result is one and the same whatever the
//     scheduling.  Bound by latency: three rounds through the cluster (30 us for 32 units of 32768
//     tokens on 4 CTAs each; on one CTA, the sums read in every pass, 96).
//   move: one warp per 16-token block with holes copies codes and scales, the sources of a block fetched two blocks
//     ahead and their places one: 43 us for 32 x 8192 slots, 230 MB at 5.3 TB/s.  The
//     layout costs that: a value token is one byte of every word of its block, so each source
//     block is read whole for a quarter of its tokens (the moved bytes alone are 16 us).
//     A key
//     token is 16-byte pieces of the fragment-native block; a value token is one
//     field (byte, nibbles or half) of every word of four lanes' pieces, merged
//     into the destination's words, which only this warp writes.
#include "kvq_decode_impl.cuh"

namespace kvq {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kWin = 8192;       // holes matched per walk; more take another walk
constexpr int kKeyCap = 32768;   // tokens whose keys stay in shared memory; longer rows read their sums again
constexpr int kBins = 2048, kReplicas = 4;
constexpr int kLoads = 8;
constexpr int kMinSpan = 2048;   // stored tokens that make another CTA of the cluster worth it (64 units of 4096: 39 us
                                 // with one CTA a unit, 37 with two)
constexpr long long kMoveCtas = 4;  // of the move an SM, two of which are resident (4 / 8 / 16: 74 / 76 / 81 us)
static_assert(kBins == 2 * kSelThreads && kReplicas * kBins <= 2 * kWin && kSelWarps == 32, "");

// What one sequence keeps: of Lq stored tokens (and the ring's), n go.
struct EvictLen {
  int L, Lq, n;
};

__device__ __forceinline__ EvictLen evict_len(const EvictArgs& a, int b, bool& bad) {
  EvictLen e;
  const int W = a.c.window;
  const int room = min(table_tokens(a.mbps, W), a.stride);
  e.L = a.seq_lens[b];
  int keep = a.keep[b];
  if (e.L < 0 || e.L > room || keep < 0) {
    bad = true;
    e.L = e.L < 0 ? 0 : min(e.L, room);
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

// Exclusive scan of v over the CTA; two barriers.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sum, int warp, int lane) {
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t n = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += n;
  }
  if (lane == 31) warp_sum[warp] = s;
  __syncthreads();
  uint32_t w = warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t n = __shfl_up_sync(kFull, w, o);
    if (lane >= o) w += n;
  }
  const uint32_t before = __shfl_sync(kFull, w, max(warp - 1, 0));
  __syncthreads();  // the sums have been read
  return s - v + (warp > 0 ? before : 0u);
}

// ---- the CTAs of one unit form a cluster and read each other's shared memory
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
  return at;
}
__device__ __forceinline__ uint2 remote_load2(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint4 remote_load4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void remote_store(uint32_t at, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// What the selection found: keys above `prefix` (after the shift) stay, and the first `need` equal ones.
struct Threshold {
  uint32_t prefix, need;
  int shift;
};

// Calls f(slot, key) for this thread's keys, eight loads in flight; every lane of a warp calls it together
// (slot < 0: none).
template <class Key, class F>
__device__ __forceinline__ void each_key(const Key& key, int from, int n, int tid, F f) {
  for (int base = from + (tid & ~31); base < n; base += kLoads * kSelThreads) {
    uint32_t k[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int s = base + i * kSelThreads + (tid & 31);
      k[i] = s < n ? key(s) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int s = base + i * kSelThreads + (tid & 31);
      if (base + i * kSelThreads < n) f(s < n ? s : -1, k[i]);
    }
  }
}

// One digit of the radix selection: `bits` bits of the keys whose upper bits are the prefix.  `first`
// reads the sums and leaves their keys in shared memory for the other passes.
template <class Key, class Put>
__device__ __forceinline__ bool select_digit(Threshold& th, int bits, const Key& key, const Put& put, int from, int to,
                                             uint32_t* hist, uint32_t* sums, uint32_t* warp_sum, uint32_t* pick, int tid,
                                             int warp, int lane) {
  for (int i = tid; i < kReplicas * kBins / 4; i += kSelThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  const int shift = th.shift - bits;
  uint32_t* mine = hist + (warp % kReplicas) * kBins;
  each_key(key, from, to, tid, [&](int s, uint32_t k) {
    put(s, k);
    const bool in = s >= 0 && (th.shift == 32 || (k >> (th.shift & 31)) == th.prefix);
    const uint32_t d = (k >> shift) & ((1u << bits) - 1u), who = __ballot_sync(kFull, in);
    if (who == 0u) return;
    // many equal digits (zeros, protected tokens) would queue on one address: one add for all of them
    const uint32_t d0 = __shfl_sync(kFull, d, __ffs(who) - 1);
    const uint32_t same = __ballot_sync(kFull, in && d == d0);
    if (in && d != d0) atomicAdd(&mine[d], 1u);
    if (lane == __ffs(who) - 1) atomicAdd(&mine[d0], uint32_t(__popc(same)));
  });
  __syncthreads();
  // thread i: bins kBins - 1 - 2i and the one below, from the top; this CTA's keys, then all of the cluster's
  const int top = kBins - 1 - 2 * tid;
  uint2 c = make_uint2(0u, 0u);
#pragma unroll
  for (int r = 0; r < kReplicas; ++r) {
    const uint2 v = *reinterpret_cast<const uint2*>(&hist[r * kBins + top - 1]);
    c.x += v.x;
    c.y += v.y;
  }
  *reinterpret_cast<uint2*>(&sums[top - 1]) = c;
  cluster_sync();
  uint32_t c0 = 0u, c1 = 0u;
  for (uint32_t r = 0, n = cluster_size(); r < n; ++r) {
    const uint2 v = remote_load2(remote(&sums[top - 1], r));
    c0 += v.y;
    c1 += v.x;
  }
  const uint32_t above = block_scan(c0 + c1, warp_sum, warp, lane);
  if (above < th.need && above + c0 + c1 >= th.need) {  // exactly one thread
    const bool second = above + c0 < th.need;
    pick[0] = top - (second ? 1 : 0);
    pick[1] = th.need - above - (second ? c0 : 0u);
    pick[2] = second ? c1 : c0;
  }
  __syncthreads();
  th.prefix = th.shift == 32 ? pick[0] : (th.prefix << bits) | pick[0];
  th.need = pick[1];
  th.shift = shift;
  return pick[2] != th.need;  // all of the digit stay: the lower digits decide nothing
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t sm[];
  uint32_t* hist = sm;                                   // [kReplicas][kBins], and after the selection:
  int* hole_list = reinterpret_cast<int*>(sm);           // [kWin] slots to fill, by rank
  int* tail_list = hole_list + kWin;                     // [kWin] tokens that fill them
  uint32_t* sums = sm + 2 * kWin;                        // [2][kBins], digits in turn: the cluster reads them
  uint32_t* warp_sum = sums + 2 * kBins;                 // [32]
  uint32_t* pick = warp_sum + 32;                        // [4]: digit, rank within it, keys of it
  uint32_t* counts = pick + 4;                           // [kSelWarps + 1][4]: the warps' runs, the CTA's
  uint32_t* keys = counts + 4 * (kSelWarps + 1);         // [a CTA's share of the stride, or kKeyCap]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = int(cluster_size()), r = int(cluster_rank()), log_c = 31 - __clz(C);
  const int H = a.c.H, u = int(blockIdx.x) >> log_c, b = u / H, h = u % H;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  bool bad = false;
  const int next_pos = a.next_pos ? a.next_pos[b] : 0;
  const EvictLen e = evict_len(a, b, bad);
  const int K = e.Lq - e.n, new_len = e.L - e.n;
  if (h == 0 && r == 0 && tid == 0) {
    a.new_lens[b] = new_len;
    if (bad) flag(a.err, KVQ_DEVERR_SEQ_LEN);
  }
  const size_t row = size_t(u) * a.stride;
  int* source = a.source + row;
  const long long from = (long long)(a.next_pos ? next_pos : e.L) - a.protect_recent;
  const RowKeys first_key{a.mass + row, a.token_pos ? a.token_pos + row : nullptr, a.protect_first,
                          int(max(from, -2147483647ll))};
  // this CTA's run of slots
  const int span = int(((long long)e.Lq + (kSelThreads << log_c) - 1) >> (10 + log_c)) * kSelThreads;
  const int c0 = int(min((long long)r * span, (long long)e.Lq)), c1 = int(min((long long)c0 + span, (long long)e.Lq));
  const bool cached = span <= kKeyCap;
  // token s keeps its slot, or moves to it from f
  auto follow = [&](int s, int f) {
    if (a.mass_out && (f != s || a.mass_out != a.mass)) a.mass_out[row + s] = a.mass[row + f];
    if (a.pos_out && (f != s || a.pos_out != a.token_pos)) a.pos_out[row + s] = a.token_pos ? a.token_pos[row + f] : f;
  };
  auto settle = [&](int s, int f) {
    source[s] = f;
    follow(s, f);
  };
  if (e.n > 0 && K > 0) {
    // ---- the K-th largest key, digits from the top
    Threshold th{0u, uint32_t(K), 32};
    auto key = [&](int s) { return cached ? keys[s - c0] : first_key(s); };
    auto none = [](int, uint32_t) {};
    auto keep_key = [&](int s, uint32_t k) {
      if (cached && s >= 0) keys[s - c0] = k;
    };
    bool more = select_digit(th, 11, first_key, keep_key, c0, c1, hist, sums, warp_sum, pick, tid, warp, lane);
    if (more) more = select_digit(th, 11, key, none, c0, c1, hist, sums + kBins, warp_sum, pick, tid, warp, lane);
    if (more) select_digit(th, 10, key, none, c0, c1, hist, sums, warp_sum, pick, tid, warp, lane);
    // ---- ranks: warp w owns a run of slots; keys above and at the threshold, below slot K and behind it
    const int per = span / kSelWarps;
    const int s0 = min(c0 + warp * per, c1), s1 = min(s0 + per, c1);
    uint32_t gb = 0u, tb = 0u, ga = 0u, ta = 0u;
    for (int base = s0; base < s1; base += 32 * kLoads) {
      uint32_t k[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) k[i] = base + i * 32 + lane < s1 ? key(base + i * 32 + lane) >> th.shift : 0u;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int s = base + i * 32 + lane;
        const bool gt = s < s1 && k[i] > th.prefix, tie = s < s1 && k[i] == th.prefix;
        gb += gt && s < K;
        tb += tie && s < K;
        ga += gt && s >= K;
        ta += tie && s >= K;
      }
    }
    gb = __reduce_add_sync(kFull, gb);
    tb = __reduce_add_sync(kFull, tb);
    ga = __reduce_add_sync(kFull, ga);
    ta = __reduce_add_sync(kFull, ta);
    uint4* const runs = reinterpret_cast<uint4*>(counts);
    if (lane == 0) runs[warp] = make_uint4(gb, tb, ga, ta);
    __syncthreads();
    const uint4 mine = runs[lane];  // lane l: warp l's run
    if (warp == 0) {
      const uint4 all = make_uint4(__reduce_add_sync(kFull, mine.x), __reduce_add_sync(kFull, mine.y),
                                   __reduce_add_sync(kFull, mine.z), __reduce_add_sync(kFull, mine.w));
      if (lane == 0) runs[kSelWarps] = all;
    }
    cluster_sync();
    const uint4 theirs = lane < C ? remote_load4(remote(&runs[kSelWarps], lane)) : make_uint4(0u, 0u, 0u, 0u);
    auto through = [&](uint32_t v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t n = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += n;
      }
      return v;
    };
    // lane l: ties, holes and kept tail tokens before run l, of runs of `width` slots from `at` that hold c;
    // of equal sums the lowest slots stay
    struct Ranks {
      uint32_t ties, holes, tails, all_holes;
    };
    auto ranks = [&](uint4 c, int at, int width, int end, uint32_t need) {
      const uint32_t ties = through(c.y + c.w) - c.y - c.w, left = need > ties ? need - ties : 0u;
      const uint32_t kb = c.x + min(c.y, left), ka = c.z + min(c.w, left - min(c.y, left));
      const long long to = min(end, K);
      const int l0 = int(min((long long)at + (long long)lane * width, to));
      const int l1 = int(min((long long)at + (long long)lane * width + width, to));
      const uint32_t nh = uint32_t(max(l1 - l0, 0)) - kb;  // an empty run holds nothing
      const uint32_t holes = through(nh), tails = through(ka);
      return Ranks{ties, holes - nh, tails - ka, __shfl_sync(kFull, holes, 31)};
    };
    const Ranks of_ctas = ranks(theirs, 0, span, e.Lq, th.need);
    const uint32_t moves = of_ctas.all_holes, ties_c = __shfl_sync(kFull, of_ctas.ties, r);
    const Ranks of_warps = ranks(mine, c0, per, c1, th.need > ties_c ? th.need - ties_c : 0u);
    const uint32_t ties0 = ties_c + __shfl_sync(kFull, of_warps.ties, warp);
    const uint32_t holes0 = __shfl_sync(kFull, of_ctas.holes, r) + __shfl_sync(kFull, of_warps.holes, warp);
    const uint32_t tails0 = __shfl_sync(kFull, of_ctas.tails, r) + __shfl_sync(kFull, of_warps.tails, warp);
    // ---- holes and the tokens that fill them, matched by rank: the ranks of a walk go to the CTAs' lists
    // 32 at a time
    const uint32_t room = uint32_t(kWin) << log_c;
    auto enlist = [&](int* list, uint32_t i, int s) {
      remote_store(remote(&list[((i >> (5 + log_c)) << 5) | (i & 31u)], (i >> 5) & uint32_t(C - 1)), s);
    };
    uint32_t w0 = 0u;
    do {
      uint32_t tr = ties0, hr = holes0 - w0, tl = tails0 - w0;  // ranks of other walks wrap beyond the room
      const uint32_t lt = (1u << lane) - 1u;
      for (int base = s0; base < s1; base += 32) {
        const int s = base + lane;
        const uint32_t k = s < s1 ? key(s) >> th.shift : 0u;
        const bool tie = s < s1 && k == th.prefix;
        const uint32_t ties_here = __ballot_sync(kFull, tie);
        const bool kept = s < s1 && (k > th.prefix || (tie && tr + __popc(ties_here & lt) < th.need));
        tr += __popc(ties_here);
        const bool hole = s < s1 && s < K && !kept, tail = s >= K && kept;
        const uint32_t hm = __ballot_sync(kFull, hole), tm = __ballot_sync(kFull, tail);
        const uint32_t hi = hr + __popc(hm & lt), ti = tl + __popc(tm & lt);
        if (hole && hi < room) enlist(hole_list, hi, s);
        if (tail && ti < room) enlist(tail_list, ti, s);
        hr += __popc(hm);
        tl += __popc(tm);
        if (w0 == 0u && kept && s < K) settle(s, s);  // in place it changes nothing
      }
      cluster_sync();
      const uint32_t m = min(moves - w0, room);
      for (int i = tid; i < kWin; i += kSelThreads) {
        if ((((uint32_t(i) >> 5) << log_c | uint32_t(r)) << 5 | (i & 31u)) >= m) break;
        source[hole_list[i]] = tail_list[i];
        if (cached) follow(hole_list[i], tail_list[i]);
      }
      w0 += room;
      cluster_sync();  // the lists have been read, and every token that moves
    } while (w0 < moves);
    if (!cached) {  // the walks read the sums again: none may be overwritten before the last one
      for (int s = r * kSelThreads + tid; s < K; s += kSelThreads << log_c)
        if (source[s] != s) follow(s, source[s]);
      cluster_sync();
    }
  } else {
    for (int s = r * kSelThreads + tid; s < K; s += kSelThreads << log_c) settle(s, s);
  }
  // the ring's tokens follow: a multiple of the window goes, so they move by it or stay, onto no entry read here
  for (int s = K + r * kSelThreads + tid; s < new_len; s += kSelThreads << log_c) settle(s, s + e.n);
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
  const int H = a.c.H, u = blockIdx.x, b = u / H, h = u % H;
  bool bad = false;
  const EvictLen e = evict_len(a, b, bad);
  const int K = e.Lq - e.n, blocks = (K + kBlock - 1) / kBlock;
  if (e.n == 0) return;
  const int* table = a.table + size_t(b) * a.mbps;
  const int* source = a.source + size_t(u) * a.stride;
  const size_t hb = size_t(h) * a.c.num_blocks;
  // the sources of a block are fetched two blocks ahead, their places one block ahead
  const int step = int(gridDim.y) * int(blockDim.x >> 5);
  auto fetch_source = [&](long long blk) {
    const long long slot = blk * kBlock + lane;
    return blk < blocks && lane < kBlock && slot < K ? source[slot] : -1;
  };
  struct Places {
    int from, to;
  };
  auto fetch_places = [&](long long blk, int src) {
    const bool hole = src >= 0 && src != blk * kBlock + lane;
    return Places{hole ? table[src / kBlock] : 0, hole ? table[blk] : 0};
  };
  long long blk = (long long)blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  int src = fetch_source(blk), src1 = fetch_source(blk + step);
  Places at = fetch_places(blk, src);
  for (int src2; blk < blocks; blk += step, src = src1, src1 = src2) {
    const Places now = at;
    at = fetch_places(blk + step, src1);
    src2 = fetch_source(blk + 2ll * step);
    bool hole = src >= 0 && src != blk * kBlock + lane;
    if (!__any_sync(kFull, hole)) continue;
    int sphys = now.from;
    if (hole && (now.from < 0 || now.from >= a.c.num_blocks || now.to < 0 || now.to >= a.c.num_blocks)) {
      flag(a.err, KVQ_DEVERR_BLOCK_ID);
      hole = false;
    }
    const uint32_t holes = __ballot_sync(kFull, hole);
    if (holes == 0u) continue;
    const int dphys = __shfl_sync(kFull, now.to, __ffs(holes) - 1);
    const int stok = src & (kBlock - 1);
    // keys: token g + 8 hi owns the pieces of lanes 4g..4g+3 in the chunks of its half
    constexpr int kPer = KB / 4;  // 512-byte chunks per half
    uint8_t* kd = a.c.k_codes + (hb + dphys) * block_bytes(KB);
    const uint8_t* kfrom[2];
    bool kmine[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tok = g + 8 * i;
      const int sp = __shfl_sync(kFull, sphys, tok), st = __shfl_sync(kFull, stok, tok);
      kmine[i] = holes >> tok & 1u;
      kfrom[i] = a.c.k_codes + (hb + (kmine[i] ? sp : 0)) * block_bytes(KB) + (st >> 3) * kPer * 512 + (4 * (st & 7) + t) * 16;
    }
    // values: lane t's pieces hold tokens 2t, 2t + 8, 2t + 1, 2t + 9
    uint8_t* vd = a.c.v_codes + (hb + dphys) * block_bytes(VB);
    const uint8_t* vfrom[4];
    int js[4];
    uint32_t vmine = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int tok = 2 * t + (j >> 1) + 8 * (j & 1);
      const int sp = __shfl_sync(kFull, sphys, tok), st = __shfl_sync(kFull, stok, tok);
      const bool mine = holes >> tok & 1u;
      vmine |= mine ? 1u << j : 0u;
      vfrom[j] = a.c.v_codes + (hb + (mine ? sp : 0)) * block_bytes(VB) + (4 * g + ((st & 7) >> 1)) * 16;
      js[j] = value_j(st);
    }
    // every load of the keys, the scales and two chunks of values is in flight before the first store
    uint4 k[2 * kPer];
#pragma unroll
    for (int c = 0; c < 2 * kPer; ++c)
      if (kmine[c / kPer]) k[c] = *reinterpret_cast<const uint4*>(kfrom[c / kPer] + c % kPer * 512);
    constexpr int kTwo = VB / 2 < 2 ? 1 : 2;
#pragma unroll
    for (int c0 = 0; c0 < VB / 2; c0 += kTwo) {
      uint4 d[kTwo], v[kTwo][4];
#pragma unroll
      for (int c = 0; c < kTwo; ++c) {
        // four new tokens fill the words: nothing of the old ones is needed
        d[c] = make_uint4(0u, 0u, 0u, 0u);
        if (vmine && vmine != 15u) d[c] = *(reinterpret_cast<const uint4*>(vd) + (c0 + c) * 32 + lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (vmine >> j & 1u) v[c][j] = *reinterpret_cast<const uint4*>(vfrom[j] + (c0 + c) * 512);
      }
      if (c0 == 0) {
#pragma unroll
        for (int c2 = 0; c2 < 2 * kPer; ++c2)
          if (kmine[c2 / kPer]) reinterpret_cast<uint4*>(kd)[c2 * 32 + lane] = k[c2];
      }
#pragma unroll
      for (int c = 0; c < kTwo; ++c) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (vmine >> j & 1u) move_field<VB>(d[c], v[c][j], j, js[j]);
        if (vmine) *(reinterpret_cast<uint4*>(vd) + (c0 + c) * 32 + lane) = d[c];
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

template <int KB, int VB>
cudaError_t launch_move(const EvictArgs& a, int sms, cudaStream_t s) {
  const int units = a.B * a.c.H;
  // one block a warp while that fills the GPU's warps once, then several
  const long long most = (a.mbps + 7ll) / 8, fill = (kMoveCtas * sms + units - 1ll) / units;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units, unsigned(most < fill ? most : fill));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel<KB, VB>, a);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int units = a.B * a.c.H;
  int c = 8;
  while (c > 1 && ((long long)units * c > sms || (long long)c * kMinSpan > a.stride)) c /= 2;
  const int span = (a.stride + c * kSelThreads - 1) / (c * kSelThreads) * kSelThreads;
  constexpr int fixed = (2 * kWin + 2 * kBins + 32 + 4 + 4 * (kSelWarps + 1)) * 4;
  e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, fixed + kKeyCap * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units * c));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = fixed + (span < kKeyCap ? span : kKeyCap) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if ((e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a)) != cudaSuccess) return e;
  const int kb = a.c.k_bits, vb = a.c.v_bits;
  if (kb == 8 && vb == 8) return launch_move<8, 8>(a, sms, s);
  if (kb == 4 && vb == 4) return launch_move<4, 4>(a, sms, s);
  if (kb == 4 && vb == 8) return launch_move<4, 8>(a, sms, s);
  if (kb == 8 && vb == 4) return launch_move<8, 4>(a, sms, s);
  if (kb == 16 && vb == 16) return launch_move<16, 16>(a, sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
