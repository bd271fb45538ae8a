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
// Moving pages is copying: a warp takes one page of one head and layer, keys, values and metadata, all its
// loads in flight before its first store.
#include "kvq_decode_impl.cuh"

namespace kvq {
namespace {

constexpr int kPageThreads = 1024;
constexpr int kPageCtas = 8;  // of the cluster
constexpr int kPageWarps = kPageCtas * kPageThreads / 32;

__device__ __forceinline__ int cluster_cta() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return int(r);
}
// All threads of the cluster; global writes before it are seen behind it (reads go to L2: __ldcg).
__device__ __forceinline__ void cluster_sync() {
  __threadfence();
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
  long long wanted = (long long)x.len + a.room;
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
  const int chunks = (width + 127) / 128, front = (a.sinks + kBlock - 1) / kBlock;
  for (int w = gwarp; w < B * chunks; w += kPageWarps) {
    const int r = w / chunks, j0 = (w % chunks) * 128 + lane;
    const Row x = rows[r];
    const int* mine = a.table + size_t(r) * width;
    const int* theirs = a.table + size_t(max(x.parent, 0)) * width;
    int old[4], now[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + 32 * k;
      old[k] = j < width ? mine[j] : -1;
      now[k] = j < width && x.parent >= 0 ? theirs[j] : -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + 32 * k;
      if (j >= width) continue;
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
  auto last_of = [&](int r, int& refs) {
    const Row x = rows[r];
    refs = 0;
    if (x.parent < 0 || (max(x.len - a.window, 0) & (kBlock - 1)) == 0) return -1;
    const int e = __ldcg(&a.table_out[size_t(r) * width + x.count - 1]);
    if (e < 0) {
      bad |= KVQ_DEVERR_BLOCK_ID;
      return -1;
    }
    refs = __ldcg(&a.refs_out[e]);
    return e;
  };
  constexpr int kPer = kMaxBatch / kPageThreads;  // rows a thread: tid * per ..
  const int per = (B + kPageThreads - 1) / kPageThreads;
  int last[kPer], held[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = tid * per + i;
    last[i] = -1;
    if (i < per && r < B) {
      last[i] = last_of(r, held[i]);
      if (last[i] >= 0 && held[i] > 1) wr.add(last[i], r);
    }
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
      ask[i] = __ldcg(&ws[kWsMissing + r]) + copy[i];
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
  // ---- free pages of this CTA's part of the pool
  const int part = ((n + kPageCtas - 1) / kPageCtas + 31) / 32 * 32;
  const int p0 = min(cta * part, n), p1 = min(p0 + part, n);
  int free_here = 0, free_cta;
  for (int i = p0 + tid; i < p1; i += kPageThreads) free_here += __ldcg(&a.refs_out[i]) == 0;
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
      const int r = w / chunks;
      for (int j = (w % chunks) * 128 + lane; j < min(width, (w % chunks) * 128 + 128); j += 32) {
        const size_t at = size_t(r) * width + j;
        const int was = a.table[at], now = __ldcg(&a.table_out[at]);
        a.table_out[at] = was;
        if (was == now) continue;
        if (was >= 0 && was < n) atomicAdd(&a.refs_out[was], 1);
        if (now >= 0) atomicAdd(&a.refs_out[now], -1);
      }
    }
    if (cta == 0) {
      for (int r = tid; r < B; r += kPageThreads) a.lens_out[r] = a.lens[r];
      if (tid == 0) {
        *a.num_copies = 0;
        flag(a.err, KVQ_DEVERR_NO_BLOCKS);
      }
    }
  } else {
    if (cta == 0) {
      for (int r = tid; r < B; r += kPageThreads) a.lens_out[r] = rows[r].len;
      if (tid == 0) *a.num_copies = all_copies;
    }
    // ---- the k-th free page goes to the k-th place that asks
    for (int base = p0; base < p1 && free_before < all_asks; base += kPageThreads) {
      const int i = base + tid;
      const bool is_free = i < p1 && __ldcg(&a.refs_out[i]) == 0;
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

// ---- copies of pages: a warp per (layer, pair, head)
__device__ __forceinline__ void copy_lines(uint8_t* dst, const uint8_t* src, int bytes, int lane) {
  const uint4* s = reinterpret_cast<const uint4*>(src) + lane;
  uint4* d = reinterpret_cast<uint4*>(dst) + lane;
  uint4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k * 512 < bytes) v[k] = s[k * 32];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k * 512 < bytes) d[k * 32] = v[k];
}

__global__ void __launch_bounds__(256) copy_blocks_kernel(const CopyArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int n = min(max(*a.num_copies, 0), a.max_copies), H = a.H, per = n * H;
  const long long all = (long long)per * a.layers;
  for (long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); w < all; w += (long long)gridDim.x * 8) {
    const int layer = int(w / per), rest = int(w % per), pair = rest / H, h = rest % H;
    const int2 m = reinterpret_cast<const int2*>(a.copies)[pair];
    if (m.x < 0 || m.y < 0 || m.x >= a.num_blocks || m.y >= a.num_blocks) {
      if (lane == 0) flag(a.err, KVQ_DEVERR_BLOCK_ID);
      continue;
    }
    const size_t src = size_t(h) * a.num_blocks + m.x, dst = size_t(h) * a.num_blocks + m.y;
    const CopyPools& p = a.pools[layer];
    copy_lines(p.k + dst * a.k_bytes, p.k + src * a.k_bytes, a.k_bytes, lane);
    copy_lines(p.v + dst * a.v_bytes, p.v + src * a.v_bytes, a.v_bytes, lane);
    if (lane * 16 < a.meta_bytes)
      *reinterpret_cast<uint4*>(p.meta + dst * a.meta_bytes + lane * 16) =
          *reinterpret_cast<const uint4*>(p.meta + src * a.meta_bytes + lane * 16);
  }
}

// ---- rings of a bf16 window: row r becomes its parent's, in place.  A CTA holds a slice of every row that changes in
// shared memory before it writes any
__global__ void __launch_bounds__(256) fork_windows_kernel(const RingArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int moved_s;
  uint16_t* to = reinterpret_cast<uint16_t*>(smem);  // [B] rows that change, and their parents
  uint16_t* from = to + a.B;
  uint4* slice = reinterpret_cast<uint4*>(smem + (a.B * 4 + 15) / 16 * 16);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) moved_s = 0;
  __syncthreads();
  for (int r = threadIdx.x; r < a.B; r += blockDim.x) {
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
  const int lines = a.slice_bytes / 16, all = moved_s * lines;
  const int slices = a.row_bytes / a.slice_bytes;
  for (int u = blockIdx.x; u < 2 * a.layers * slices; u += gridDim.x) {
    uint8_t* ring = (u / slices % 2 ? a.rings[u / slices / 2].v : a.rings[u / slices / 2].k) +
                    size_t(u % slices) * a.slice_bytes;
    for (int i = threadIdx.x; i < all; i += blockDim.x)
      slice[i] = reinterpret_cast<const uint4*>(ring + size_t(from[i / lines]) * a.row_bytes)[i % lines];
    __syncthreads();
    for (int i = threadIdx.x; i < all; i += blockDim.x)
      reinterpret_cast<uint4*>(ring + size_t(to[i / lines]) * a.row_bytes)[i % lines] = slice[i];
    __syncthreads();
  }
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
  const int smem = update_smem(a.B);
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  void* args[] = {&a};
  return launch(k, dim3(kPageCtas), kPageThreads, smem, s, args);
}

cudaError_t launch_pages_compact(PagesArgs a, cudaStream_t s) {
  void* args[] = {&a};
  return launch(reinterpret_cast<const void*>(pages_compact_kernel), dim3(kPageCtas), kPageThreads, 0, s, args);
}

cudaError_t launch_copy_blocks(CopyArgs a, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long ctas = ((long long)a.max_copies * a.H * a.layers + 7) / 8;
  void* args[] = {&a};
  return launch(reinterpret_cast<const void*>(copy_blocks_kernel), dim3(unsigned(ctas < 4ll * sms ? ctas : 4ll * sms)), 256,
                0, s, args);
}

cudaError_t launch_fork_windows(RingArgs a, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // slices as wide as 64 KB of shared memory hold for every row, from 16 bytes (4096 rows) to 4 KB
  a.slice_bytes = 4096;
  while (a.slice_bytes > 16 && a.slice_bytes * a.B > 65536) a.slice_bytes /= 2;
  const void* k = reinterpret_cast<const void*>(fork_windows_kernel);
  const int smem = (a.B * 4 + 15) / 16 * 16 + a.B * a.slice_bytes;
  if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
  const long long units = 2ll * a.layers * (a.row_bytes / a.slice_bytes);
  void* args[] = {&a};
  return launch(k, dim3(unsigned(units < 2ll * sms ? units : 2ll * sms)), 256, smem, s, args);
}

}  // namespace kvq
