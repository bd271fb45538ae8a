// Pages of a cache on the device: kvq_pages_update, kvq_pages_compact, kvq_copy_blocks, kvq_fork_windows.
//
// A page is a 16-token block of every layer's pools under one number; refs[i] counts the table entries that
// hold page i (and its user's own claims), 0 means free.
//
// Update and compaction decide about pages: integers, whose result is one and the same whatever the
// scheduling (free pages go out from the lowest on, in the order of rows).  Each is one launch of one cluster of
// 8 CTAs: the steps need the whole batch's counts in between, and a cluster barrier costs less than a
// launch.  Both are bound by latency, a chain of reads from L2 between barriers.
//
// Moving pages is copying: a warp takes pages of one head and layer in turn, and its lane 0 moves keys, values and
// metadata by bulk copies through a ring of places in shared memory, a page out as soon as it has landed.
#include "kvq_decode_impl.cuh"

namespace kvq {
namespace {

constexpr int kPageThreads = 1024;
constexpr int kPageCtas = 8;  // of the cluster
constexpr int kPageWarps = kPageCtas * kPageThreads / 32;
constexpr int kKeep = 16;  // pages of a thread whose counts stay in registers (pools of 131072)
constexpr int kCols = 8;  // table entries of a lane in flight (64 rows of 2048: 4 18.2 us, 8 and 16 16.5; 48 rows of 300: 16.4, 16.5, 18.6)

__device__ __forceinline__ int cluster_cta() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return int(r);
}
// All threads of the cluster; the cluster's global writes before it are seen behind it (release and acquire at cluster
// scope; what other CTAs write is read from L2, __ldcg).
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Inclusive scan of v over the CTA's 1024 threads, and the sum of all; two barriers.
__device__ __forceinline__ int cta_scan(int v, int* warp_sum, int& total, int warp, int lane) {
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += n;
  }
  if (lane == 31) warp_sum[warp] = s;
  __syncthreads();
  int w = warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(kFull, w, o);
    if (lane >= o) w += n;
  }
  total = __shfl_sync(kFull, w, 31);
  const int before = __shfl_sync(kFull, w, max(warp - 1, 0));
  __syncthreads();
  return s + (warp > 0 ? before : 0);
}

// Workspace, in ints: counters of the CTAs, missing pages of each row, and the new place of each page (compaction).
constexpr int kWsCounts = 0, kWsAny = kPageCtas, kWsMissing = 64, kWsMap = kWsMissing + kMaxBatch;

// What becomes of row r: its parent row (-1: freed), tokens, blocks that hold some, blocks that it asks for.
struct Row {
  int parent, len, count, need;
};

__device__ __forceinline__ Row row_of(const PagesArgs& a, int r, uint32_t& bad) {
  Row x{a.parent ? a.parent[r] : r, 0, 0, 0};
  if (x.parent < -1 || x.parent >= a.B) {
    bad |= KVQ_DEVERR_POSITION;
    x.parent = r;
  }
  if (x.parent < 0) return x;
  const int most = table_tokens(a.width, a.window);
  x.len = a.lens[x.parent];
  if (x.len < 0 || x.len > most) {
    bad |= KVQ_DEVERR_SEQ_LEN;
    x.len = x.len < 0 ? 0 : most;
  }
  int room = a.rooms ? a.rooms[r] : a.room;
  if (room < 0) {
    bad |= KVQ_DEVERR_SEQ_LEN;
    room = 0;
  }
  long long wanted = (long long)x.len + room;
  if (wanted > most) {
    bad |= KVQ_DEVERR_SEQ_LEN;
    wanted = most;
  }
  x.count = (max(x.len - a.window, 0) + kBlock - 1) / kBlock;
  x.need = (max(int(wanted) - a.window, 0) + kBlock - 1) / kBlock;
  return x;
}

__device__ __forceinline__ bool page_ok(const PagesArgs& a, int page, uint32_t& bad) {
  if (page < 0 || page >= a.num_blocks) {
    if (page != -1) bad |= KVQ_DEVERR_BLOCK_ID;
    return false;
  }
  return true;
}

// The rows that write to a page that others hold, by page.
struct Writers {
  int* page;   // [slots], -1: none
  int* rows;   // how many
  int* first;  // the lowest
  int mask;
  __device__ __forceinline__ int find(int p) const {
    int i = int((uint32_t(p) * 2654435761u) >> 7) & mask;
    while (page[i] != p) i = (i + 1) & mask;
    return i;
  }
  __device__ __forceinline__ void add(int p, int r) const {
    int i = int((uint32_t(p) * 2654435761u) >> 7) & mask;
    for (;;) {  // at most half of the slots are taken
      const int was = atomicCAS(&page[i], -1, p);
      if (was == -1 || was == p) break;
      i = (i + 1) & mask;
    }
    atomicAdd(&rows[i], 1);
    atomicMin(&first[i], r);
  }
};

__host__ __device__ inline int writer_slots(int B) {
  int n = 32;
  while (n < 2 * B) n *= 2;
  return n;
}

__host__ __device__ inline int update_smem(int B) {
  return B * int(sizeof(Row)) + (2 * B + 4) * 4 + 3 * writer_slots(B) * 4;
}

// Shared memory of fork_windows_kernel, whose slices are as wide as 52 KB each hold for every row.
__host__ inline int ring_slice(int B) {
  int bytes = 4096;
  while (bytes > 16 && bytes * B > 53248) bytes /= 2;
  return bytes;
}
__host__ inline int ring_smem(int B) { return (B * 4 + 15) / 16 * 16 + 2 * B * ring_slice(B); }

__global__ void __launch_bounds__(kPageThreads) __cluster_dims__(kPageCtas, 1, 1) pages_update_kernel(const PagesArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int warp_sum[32];
  const int B = a.B, width = a.width, n = a.num_blocks;
  Row* rows = reinterpret_cast<Row*>(smem);
  int* pages_before = reinterpret_cast<int*>(rows + B);  // [B + 1] pages that the rows before r ask for
  int* copies_before = pages_before + B + 1;             // [B + 1]
  const int slots = writer_slots(B);
  Writers wr{copies_before + B + 3, nullptr, nullptr, slots - 1};
  wr.rows = wr.page + slots;
  wr.first = wr.rows + slots;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = cluster_cta();
  const int gwarp = cta * 32 + warp, gtid = cta * kPageThreads + tid;
  int* ws = a.ws;
  uint32_t bad = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  for (int r = tid; r < B; r += kPageThreads) rows[r] = row_of(a, r, bad);
  for (int i = tid; i < slots; i += kPageThreads) {
    wr.page[i] = -1;
    wr.rows[i] = 0;
    wr.first[i] = 0x7fffffff;
  }
  if (a.refs_out != a.refs)
    for (int i = gtid; i < n; i += kPageCtas * kPageThreads) a.refs_out[i] = a.refs[i];
  if (gtid == 0) ws[kWsAny] = 0;
  cluster_sync();

  // ---- every row takes its parent's pages: those that hold tokens, but for those between the sinks and the window,
  // and its own that were kept for coming ones
  // (no sum passes 32 bits: width may be 2^31 - 1, and so may the sinks, which are cut to what a row can hold)
  const int chunks = (width - 1) / (32 * kCols) + 1;
  const int front = (min(a.sinks, table_tokens(width, a.window)) + kBlock - 1) / kBlock;
  for (int w = gwarp; w < B * chunks; w += kPageWarps) {
    const int r = w / chunks, j0 = (w % chunks) * 32 * kCols + lane;
    const Row x = rows[r];
    const int* mine = a.table + size_t(r) * width;
    const int* theirs = a.table + size_t(max(x.parent, 0)) * width;
    int old[kCols], now[kCols];
#pragma unroll
    for (int k = 0; k < kCols; ++k) {
      const int j = j0 + 32 * k;
      old[k] = j < width ? mine[j] : -1;
      now[k] = j < width && x.parent >= 0 ? theirs[j] : -1;
    }
#pragma unroll
    for (int k = 0; k < kCols; ++k) {
      const int j = j0 + 32 * k;
      if (j >= width) break;
      const bool held = j < x.count ? a.span == 0 || j < front || (j + 1) * kBlock > x.len - a.span
                                    : x.parent == r && j < x.need;
      if (!page_ok(a, old[k], bad)) old[k] = -1;
      if (!held || !page_ok(a, now[k], bad)) now[k] = -1;
      a.table_out[size_t(r) * width + j] = now[k];
      if (old[k] != now[k]) {
        if (old[k] >= 0) atomicAdd(&a.refs_out[old[k]], -1);
        if (now[k] >= 0) atomicAdd(&a.refs_out[now[k]], 1);
      }
    }
  }
  cluster_sync();

  // ---- pages for coming tokens: entry -2 - i where the row's i-th one is missing.  One that others hold (a row was cut
  // back to fewer tokens) is not to be written to: missing too
  bool any = false;
  for (int r = gwarp; r < B; r += kPageWarps) {
    const Row x = rows[r];
    int missing = 0;
    for (int j0 = x.count; j0 < x.need; j0 += 32) {
      const int j = j0 + lane;
      bool gone = false;
      if (j < x.need) {
        const int e = __ldcg(&a.table_out[size_t(r) * width + j]);
        gone = e < 0;
        if (e >= 0 && __ldcg(&a.refs_out[e]) > 1) gone = any = true;
      }
      const uint32_t who = __ballot_sync(kFull, gone);
      if (gone) a.table_out[size_t(r) * width + j] = -2 - (missing + __popc(who & ((1u << lane) - 1u)));
      missing += __popc(who);
    }
    if (lane == 0) ws[kWsMissing + r] = missing;
  }
  if (any) ws[kWsAny] = 1;
  cluster_sync();
  // what is read next, on its way together with the word that says whether it is final
  constexpr int kPer = kMaxBatch / kPageThreads;  // rows a thread: tid * per ..
  const int per = (B + kPageThreads - 1) / kPageThreads;
  int last[kPer], held[kPer], gone[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = tid * per + i;
    last[i] = -1;
    gone[i] = 0;
    if (i < per && r < B) {
      const Row x = rows[r];
      gone[i] = __ldcg(&ws[kWsMissing + r]);
      if (x.parent >= 0 && (max(x.len - a.window, 0) & (kBlock - 1)) != 0) {
        last[i] = __ldcg(&a.table_out[size_t(r) * width + x.count - 1]);
        if (last[i] < 0) bad |= KVQ_DEVERR_BLOCK_ID;
      }
    }
  }
  if (__ldcg(&ws[kWsAny])) {
    for (int r = gwarp; r < B; r += kPageWarps) {
      const Row x = rows[r];
      if (x.parent != r) continue;
      for (int j = x.count + lane; j < x.need; j += 32) {
        const int was = a.table[size_t(r) * width + j];
        if (was >= 0 && was < n && __ldcg(&a.table_out[size_t(r) * width + j]) < 0) atomicAdd(&a.refs_out[was], -1);
      }
    }
    cluster_sync();
  }

  // ---- each row's last page, where it has room left: its own alone, or to be copied.  Of the rows that write to it the
  // lowest keeps it, if no one else holds it.  Every CTA finds this for all rows
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (last[i] >= 0) {
      held[i] = __ldcg(&a.refs_out[last[i]]);
      if (held[i] > 1) wr.add(last[i], tid * per + i);
    }
  // ---- free pages of this CTA's part of the pool: a small part's counts stay in registers
  const int part = ((n + kPageCtas - 1) / kPageCtas + 31) / 32 * 32;
  const int p0 = min(cta * part, n), p1 = min(p0 + part, n);
  const bool kept = part <= kKeep * kPageThreads;
  uint32_t free_bits = 0;
  int free_here = 0, free_cta;
  if (kept) {
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const int i = p0 + k * kPageThreads + tid;
      if (i < p1 && __ldcg(&a.refs_out[i]) == 0) free_bits |= 1u << k;
    }
    free_here = __popc(free_bits);
  } else {
    for (int i = p0 + tid; i < p1; i += kPageThreads) free_here += __ldcg(&a.refs_out[i]) == 0;
  }
  __syncthreads();
  int asks = 0, copies = 0, ask[kPer], copy[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = tid * per + i;
    ask[i] = copy[i] = 0;
    if (i < per && r < B) {
      if (last[i] >= 0 && held[i] > 1) {
        const int s = wr.find(last[i]);
        copy[i] = !(wr.rows[s] == held[i] && wr.first[s] == r);
      }
      ask[i] = gone[i] + copy[i];
      asks += ask[i];
      copies += copy[i];
    }
  }
  int all_asks, all_copies;
  int ask_at = cta_scan(asks, warp_sum, all_asks, warp, lane) - asks;
  int copy_at = cta_scan(copies, warp_sum, all_copies, warp, lane) - copies;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = tid * per + i;
    if (i < per && r < B) {
      pages_before[r] = ask_at;
      copies_before[r] = copy_at;
      ask_at += ask[i];
      copy_at += copy[i];
    }
  }
  if (tid == 0) {
    pages_before[B] = all_asks;
    copies_before[B] = all_copies;
  }
  cta_scan(free_here, warp_sum, free_cta, warp, lane);
  if (tid == 0) ws[kWsCounts + cta] = free_cta;
  cluster_sync();
  int free_before = 0, free_all = 0;
#pragma unroll
  for (int c = 0; c < kPageCtas; ++c) {
    const int f = __ldcg(&ws[kWsCounts + c]);
    free_all += f;
    free_before += c < cta ? f : 0;
  }

  if (all_asks > free_all) {
    // ---- too few: all is as it was before
    for (int w = gwarp; w < B * chunks; w += kPageWarps) {
      const int r = w / chunks, j0 = (w % chunks) * 32 * kCols;
      for (int j = j0 + lane; j < min(width, j0 + 32 * kCols); j += 32) {
        const size_t at = size_t(r) * width + j;
        const int was = a.table[at], now = __ldcg(&a.table_out[at]);
        a.table_out[at] = was;
        if (was == now) continue;
        if (was >= 0 && was < n) atomicAdd(&a.refs_out[was], 1);
        if (now >= 0) atomicAdd(&a.refs_out[now], -1);
      }
    }
    if (cta == 0) {
      for (int r = tid; r < B; r += kPageThreads) {
        a.lens_out[r] = a.lens[r];
        if (a.parent_out) a.parent_out[r] = r;
      }
      if (tid == 0) {
        *a.num_copies = 0;
        flag(a.err, KVQ_DEVERR_NO_BLOCKS);
      }
    }
  } else {
    if (cta == 0) {
      for (int r = tid; r < B; r += kPageThreads) {
        a.lens_out[r] = rows[r].len;
        if (a.parent_out) a.parent_out[r] = rows[r].parent;
      }
      if (tid == 0) *a.num_copies = all_copies;
    }
    // ---- the k-th free page goes to the k-th place that asks
    for (int base = p0; base < p1 && free_before < all_asks; base += kPageThreads) {
      const int i = base + tid;
      const bool is_free = kept ? (free_bits & 1u) != 0 : i < p1 && __ldcg(&a.refs_out[i]) == 0;
      free_bits >>= 1;
      int here;
      const int k = free_before + cta_scan(is_free ? 1 : 0, warp_sum, here, warp, lane) - 1;
      free_before += here;
      if (!is_free || k >= all_asks) continue;
      int lo = 0, hi = B - 1;  // the last row with pages_before <= k asks for it
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pages_before[mid] <= k) lo = mid;
        else hi = mid - 1;
      }
      const int r = lo, copies_here = copies_before[r + 1] - copies_before[r], m = k - pages_before[r] - copies_here;
      const Row x = rows[r];
      a.refs_out[i] = 1;
      if (m < 0) {
        const size_t at = size_t(r) * width + x.count - 1;
        const int from = __ldcg(&a.table_out[at]);
        reinterpret_cast<int2*>(a.copies)[copies_before[r]] = make_int2(from, i);
        a.table_out[at] = i;
        atomicAdd(&a.refs_out[from], -1);
      } else {
        // its place carries its number; others of the row are filled meanwhile
        for (int j = x.count + m; j < x.need; ++j)
          if (__ldcg(&a.table_out[size_t(r) * width + j]) == -2 - m) {
            a.table_out[size_t(r) * width + j] = i;
            break;
          }
      }
    }
  }
  if (bad) flag(a.err, bad);
}

// ---- compaction: live pages fill the front of the pool; the i-th free page among the first `live` takes the i-th live
// one from behind
__global__ void __launch_bounds__(kPageThreads) __cluster_dims__(kPageCtas, 1, 1) pages_compact_kernel(const PagesArgs a) {
  __shared__ int warp_sum[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = cluster_cta();
  const int gtid = cta * kPageThreads + tid, n = a.num_blocks;
  constexpr int kAll = kPageCtas * kPageThreads;
  int* ws = a.ws;
  int* map = ws + kWsMap;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int part = ((n + kPageCtas - 1) / kPageCtas + 31) / 32 * 32;
  const int p0 = min(cta * part, n), p1 = min(p0 + part, n);
  int mine = 0, total;
  for (int i = p0 + tid; i < p1; i += kPageThreads) mine += a.refs[i] > 0;
  cta_scan(mine, warp_sum, total, warp, lane);
  if (tid == 0) ws[kWsCounts + cta] = total;
  cluster_sync();
  int live = 0, before = 0, before_edge = 0, edge_cta = 0;
#pragma unroll
  for (int c = 0; c < kPageCtas; ++c) {
    before += c < cta ? __ldcg(&ws[kWsCounts + c]) : 0;
    live += __ldcg(&ws[kWsCounts + c]);
  }
  edge_cta = min(live / part, kPageCtas - 1);
#pragma unroll
  for (int c = 0; c < kPageCtas; ++c) before_edge += c < edge_cta ? __ldcg(&ws[kWsCounts + c]) : 0;
  // live pages among the first `live`: those of the parts before, and the front of the part that the edge is in
  mine = 0;
  for (int i = edge_cta * part + tid; i < live; i += kPageThreads) mine += __ldcg(&a.refs[i]) > 0;
  cta_scan(mine, warp_sum, total, warp, lane);
  const int stay = before_edge + total, moves = live - stay;
  int seen = before;  // live pages before this chunk
  for (int base = p0; base < p1; base += kPageThreads) {
    const int i = base + tid;
    const int refs = i < p1 ? __ldcg(&a.refs[i]) : 0;
    const bool on = refs > 0;
    int here;
    const int upto = seen + cta_scan(on ? 1 : 0, warp_sum, here, warp, lane);
    seen += here;
    if (i >= p1) continue;
    if (i < live && !on) a.copies[2 * (i + 1 - upto - 1) + 1] = i;  // i + 1 - upto: free ones so far
    if (i >= live) {
      if (on) a.copies[2 * (upto - stay - 1)] = i;
      else map[i] = -1;
    }
    if ((i < live) == on && a.refs_out != a.refs) a.refs_out[i] = refs;  // stays where it is
  }
  cluster_sync();
  for (int k = gtid; k < moves; k += kAll) {
    const int2 m = __ldcg(reinterpret_cast<const int2*>(a.copies) + k);
    a.refs_out[m.y] = __ldcg(&a.refs[m.x]);
    a.refs_out[m.x] = 0;
    map[m.x] = m.y;
  }
  if (gtid == 0) {
    a.num_copies[0] = moves;
    a.num_copies[1] = live;
  }
  cluster_sync();
  uint32_t bad = 0;
  const long long entries = (long long)a.B * a.width;
  for (long long base = gtid; base < entries; base += 4 * kAll) {
    int e[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = base + k * kAll < entries ? a.table[base + k * kAll] : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (base + k * kAll >= entries) continue;
      if (page_ok(a, e[k], bad) && e[k] >= live) {
        const int to = __ldcg(&map[e[k]]);
        if (to >= 0) e[k] = to;
        else bad |= KVQ_DEVERR_BLOCK_ID;  // an entry that holds a free page
      }
      a.table_out[base + k * kAll] = e[k];
    }
  }
  if (bad) flag(a.err, bad);
}

// ---- copies of pages: a warp takes (layer, pair, head) in turn, and its lane 0 moves each by bulk copies
// through shared memory: keys, values and metadata in, and out as soon as they have landed, kCopySlots of them on their way.
constexpr int kCopyWarps = 8, kCopySlots = 6;

__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

__global__ void __launch_bounds__(kCopyWarps * 32) copy_blocks_kernel(const CopyArgs a, int slots) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kCopyWarps][kCopySlots];
  __shared__ int2 places[kCopyWarps][kCopySlots];  // where a slot's page goes: layer, block in its pool
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) {
    for (int s = 0; s < kCopySlots; ++s) mbar_init(&bars[warp][s], 1);
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n = min(max(*a.num_copies, 0), a.max_copies), H = a.H;
  const uint32_t per = uint32_t(n) * H, all = per * a.layers, step = gridDim.x * kCopyWarps;
  const uint32_t kb = a.k_bytes, vb = a.v_bytes, mb = a.meta_bytes;
  uint8_t* buf = smem + size_t(warp) * slots * (kb + vb + mb);
  const uint64_t pol = l2_evict_first_policy();
  const uint32_t first = blockIdx.x * kCopyWarps + warp;
  const int mine = first < all ? int((all - 1 - first) / step) + 1 : 0;  // items of this warp
  // lane l: item base + l of the warp's; its layer, or -1 for a pair out of range, and its blocks in a pool
  int layer = -1;
  uint32_t src = 0, dst = 0;
  auto look_up = [&](int base) {
    if (base + lane >= mine) return;
    const uint32_t w = first + uint32_t(base + lane) * step, rest = w % per, pair = rest % uint32_t(n), h = rest / uint32_t(n);
    const int2 m = reinterpret_cast<const int2*>(a.copies)[pair];
    layer = m.x >= 0 && m.y >= 0 && m.x < a.num_blocks && m.y < a.num_blocks ? int(w / per) : -1;
    src = h * a.num_blocks + m.x;
    dst = h * a.num_blocks + m.y;
  };
  // the loads run slots - 1 items ahead of the stores; a slot is loaded again once its store has read it
  bool ok = true;
  int in = 0;
  for (int out = 0; out < mine && ok; ++out) {
    while (in < mine && in - out < slots - 1) {
      if (in % 32 == 0) look_up(in);
      const int s = in % slots, l = __shfl_sync(kFull, layer, in & 31);
      const uint32_t from = __shfl_sync(kFull, src, in & 31), to = __shfl_sync(kFull, dst, in & 31);
      if (lane == 0) {
        // the slot's last store has read it: at most the one after it is still on its way (in - out is slots - 2 at most)
        if (in >= slots) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        places[warp][s] = make_int2(l, int(to));
        uint8_t* at = buf + s * (kb + vb + mb);
        if (l >= 0) {
          const CopyPools& p = a.pools[l];
          mbar_arrive_expect_tx(&bars[warp][s], kb + vb + mb);
          bulk_g2s(at, p.k + size_t(from) * kb, kb, &bars[warp][s], pol);
          bulk_g2s(at + kb, p.v + size_t(from) * vb, vb, &bars[warp][s], pol);
          if (mb) bulk_g2s(at + kb + vb, p.meta + size_t(from) * mb, mb, &bars[warp][s], pol);
        } else {
          flag(a.err, KVQ_DEVERR_BLOCK_ID);
          mbar_arrive(&bars[warp][s]);
        }
      }
      __syncwarp();
      ++in;
    }
    if (lane == 0) {
      const int s = out % slots;
      ok = mbar_wait(&bars[warp][s], uint32_t(out / slots) & 1u);
      const int2 to = places[warp][s];
      if (ok && to.x >= 0) {
        const CopyPools& p = a.pools[to.x];
        const uint8_t* at = buf + s * (kb + vb + mb);
        bulk_s2g(p.k + size_t(uint32_t(to.y)) * kb, at, kb);
        bulk_s2g(p.v + size_t(uint32_t(to.y)) * vb, at + kb, vb);
        if (mb) bulk_s2g(p.meta + size_t(uint32_t(to.y)) * mb, at + kb + vb, mb);
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      if (!ok) {  // the other loads on their way land first
        flag(a.err, KVQ_DEVERR_TIMEOUT);
        for (int k = out + 1; k < in; ++k) mbar_wait(&bars[warp][k % slots], uint32_t(k / slots) & 1u);
      }
    }
    ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ---- rings of a bf16 window: row r becomes its parent's, in place.  A CTA holds a slice of every row that changes in
// shared memory before it writes any: bulk copies of a row each, the next slice on its way in while one goes out.
// (48 rows, 36 of them changed, of 8 layers, 240 MB: 16 bytes a thread by cp.async 61 us, one at a time 112.)
__global__ void __launch_bounds__(256) fork_windows_kernel(const RingArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int moved_s;
  __shared__ uint64_t bars[2];
  uint16_t* to = reinterpret_cast<uint16_t*>(smem);  // [B] rows that change, and their parents
  uint16_t* from = to + a.B;
  uint8_t* slices = smem + (a.B * 4 + 15) / 16 * 16;  // two of [B][slice_bytes]
  const int tid = threadIdx.x;
  if (tid == 0) {
    moved_s = 0;
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  for (int r = tid; r < a.B; r += blockDim.x) {
    const int p = a.parent[r];
    if (p < -1 || p >= a.B) {
      if (blockIdx.x == 0) flag(a.err, KVQ_DEVERR_POSITION);
    } else if (p >= 0 && p != r) {
      const int i = atomicAdd(&moved_s, 1);
      to[i] = uint16_t(r);
      from[i] = uint16_t(p);
    }
  }
  __syncthreads();
  const int moved = moved_s, per_pool = a.row_bytes / a.slice_bytes;
  if (moved == 0) return;
  const long long units = 2ll * a.layers * per_pool;
  const uint64_t pol = l2_evict_first_policy();
  auto ring_of = [&](long long u) {
    const int pool = int(u / per_pool);
    return (pool % 2 ? a.rings[pool / 2].v : a.rings[pool / 2].k) + size_t(u % per_pool) * a.slice_bytes;
  };
  auto load = [&](long long u, int at) {
    const uint8_t* ring = ring_of(u);
    uint8_t* slice = slices + size_t(at) * a.B * a.slice_bytes;
    if (tid == 0) mbar_arrive_expect_tx(&bars[at], uint32_t(moved) * a.slice_bytes);
    for (int i = tid; i < moved; i += blockDim.x)
      bulk_g2s(slice + size_t(i) * a.slice_bytes, ring + size_t(from[i]) * a.row_bytes, a.slice_bytes, &bars[at], pol);
  };
  int k = 0;
  if ((long long)blockIdx.x < units) load(blockIdx.x, 0);
  for (long long u = blockIdx.x; u < units; u += gridDim.x, ++k) {
    const int at = k & 1;
    if (u + gridDim.x < units) {
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // this thread's stores have read the other slice,
      __syncthreads();                                               // and so have all threads'
      load(u + gridDim.x, at ^ 1);
    }
    // every row's slice is here before any is written
    if (__syncthreads_or(!mbar_wait(&bars[at], uint32_t(k >> 1) & 1u))) {
      if (tid == 0) flag(a.err, KVQ_DEVERR_TIMEOUT);
      mbar_wait(&bars[at], uint32_t(k >> 1) & 1u);  // what is on its way lands first
      if (u + gridDim.x < units) mbar_wait(&bars[at ^ 1], uint32_t((k + 1) >> 1) & 1u);
      break;
    }
    uint8_t* ring = ring_of(u);
    const uint8_t* slice = slices + size_t(at) * a.B * a.slice_bytes;
    for (int i = tid; i < moved; i += blockDim.x)
      bulk_s2g(ring + size_t(to[i]) * a.row_bytes, slice + size_t(i) * a.slice_bytes, a.slice_bytes);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

cudaError_t launch(const void* kernel, dim3 grid, int threads, int smem, cudaStream_t s, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t sm_count(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace

size_t pages_workspace_bytes(int num_blocks) { return (size_t(kWsMap) + num_blocks) * 4; }

cudaError_t launch_pages_update(PagesArgs a, cudaStream_t s) {
  const void* k = reinterpret_cast<const void*>(pages_update_kernel);
  // the most that any call takes: another thread's call sets the same between this and the launch
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, update_smem(kMaxBatch));
  if (e != cudaSuccess) return e;
  void* args[] = {&a};
  return launch(k, dim3(kPageCtas), kPageThreads, update_smem(a.B), s, args);
}

cudaError_t launch_pages_compact(PagesArgs a, cudaStream_t s) {
  void* args[] = {&a};
  return launch(reinterpret_cast<const void*>(pages_compact_kernel), dim3(kPageCtas), kPageThreads, 0, s, args);
}

cudaError_t launch_copy_blocks(CopyArgs a, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const void* k = reinterpret_cast<const void*>(copy_blocks_kernel);
  const int item = a.k_bytes + a.v_bytes + a.meta_bytes;
  int slots = kCopySlots;  // fewer of larger pages: three of 8 KB (bf16)
  while (kCopyWarps * slots * item > 208 * 1024) --slots;
  const int smem = kCopyWarps * slots * item;
  if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 1024)) != cudaSuccess) return e;
  const long long ctas = ((long long)a.max_copies * a.H * a.layers + kCopyWarps - 1) / kCopyWarps;
  // int8 pages: 203 KB of shared memory, one CTA an SM; smaller ones several
  const int room = 227 * 1024 / (smem + 1024), most = sms * (room < 1 ? 1 : room > 3 ? 3 : room);
  void* args[] = {&a, &slots};
  return launch(k, dim3(unsigned(ctas < most ? ctas : most)), kCopyWarps * 32, smem, s, args);
}

cudaError_t launch_fork_windows(RingArgs a, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  a.slice_bytes = ring_slice(a.B);  // 16 bytes (above 1664 rows: 64 KB at 4096) to 4 KB
  const void* k = reinterpret_cast<const void*>(fork_windows_kernel);
  const int smem = ring_smem(a.B);
  // the most that any call takes, as above: no smaller number of rows takes more than kMaxBatch of them
  if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_smem(kMaxBatch))) != cudaSuccess) return e;
  const long long units = 2ll * a.layers * (a.row_bytes / a.slice_bytes);
  void* args[] = {&a};
  const int room = 224 * 1024 / (smem + 1024), most = sms * (room < 1 ? 1 : room > 4 ? 4 : room);
  return launch(k, dim3(unsigned(units < most ? units : most)), 256, smem, s, args);
}

}  // namespace kvq
