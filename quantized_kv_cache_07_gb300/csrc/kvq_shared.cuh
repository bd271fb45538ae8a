// Work split of the shared prefix (kvq_decode_shared), common to the prefix
// kernels and the merge.
//
// A unit is a tile of TQ query vectors of one group (vector v = row * G + head of
// the group) and one KV head; it has blocks[g] 16-token blocks.  Units are
// ordered by (group, tile, head); their blocks form one range of T blocks that
// the CTAs cut evenly, in steps of `step` blocks.
//
// Launches: suffix, prefix, merge, each with programmatic serialisation.  The suffix waits for the
// kernels before it and then lets the prefix kernel start, which runs beside it: their records lie apart,
// and what it reads was complete when the suffix's wait ended (its own reads of it bypass L1).  It
// waits for the suffix only before it ends, so that the merge, which waits for it, follows both.
// The wait instruction promises the writes of the grid that it waits for to the threads that have executed it.  The
// prefix kernel (and the merge, for the groups) reads what kernels before the suffix wrote without having executed it,
// and relies on two things beyond that promise: that a grid whose end another grid has waited for has its writes in L2,
// and that a CTA which starts after every suffix CTA has let it start reads L2 after that.  So every such read goes to
// L2: ld.global.cg, or a bulk copy.
#pragma once

#include "kvq_decode_impl.cuh"

namespace kvq {
namespace {

// Groups of sequences that share a prefix, in shared memory: group i holds
// sequences start[i]..start[i + 1] - 1, which share their first blocks[i] blocks.
struct GroupGeo {
  int start[kMaxGroups + 4];
  int blocks[kMaxGroups];
};

// Read and clean the caller's arrays (all threads of the CTA; ends with a
// barrier): starts within [0, B] and not falling, prefixes within the table.
// Returns (in every thread) the error bits of what had to be cleaned.
__device__ __forceinline__ unsigned load_groups(GroupGeo* geo, const int* start, const int* blocks, int n, int B,
                                                int mbps, int tid, int threads) {
  unsigned bad = 0u;
  for (int i = tid; i < n; i += threads) {
    const int p = __ldcg(blocks + i);
    if (p < 0 || p > mbps) bad |= KVQ_DEVERR_SEQ_LEN;
    geo->blocks[i] = min(max(p, 0), table_tokens(mbps, 0) / kBlock);  // behind it lies no token
  }
  if (tid < 32) {
    int top = 0;
    for (int base = 0; base <= n; base += 32) {
      const int i = base + tid;
      const int raw = i <= n ? __ldcg(start + i) : 0;
      int v = max(i <= n ? min(raw, B) : 0, 0);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int m = __shfl_up_sync(kFull, v, o);
        if (tid >= o) v = max(v, m);
      }
      v = max(v, top);
      if (i <= n) {
        if (v != raw) bad |= KVQ_DEVERR_POSITION;
        geo->start[i] = v;
      }
      top = __shfl_sync(kFull, v, 31);
    }
  }
  unsigned all = __syncthreads_or(bad & KVQ_DEVERR_SEQ_LEN) ? KVQ_DEVERR_SEQ_LEN : 0u;
  return all | (__syncthreads_or(bad & KVQ_DEVERR_POSITION) ? KVQ_DEVERR_POSITION : 0u);
}

// The group of sequence b, or -1: the last group that starts at or before b and holds it.
__device__ __forceinline__ int group_of(const GroupGeo* geo, int n, int b) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (geo->start[mid] <= b) lo = mid;
    else hi = mid - 1;
  }
  return b >= geo->start[lo] && b < geo->start[lo + 1] ? lo : -1;
}

struct SharedGeo {
  GroupGeo g;
  int unit0[kMaxGroups + 4];       // units of the groups before group i
  long long x0[kMaxGroups + 2];    // block steps of the groups before group i
  long long T;
  int units;
};

__device__ __forceinline__ int steps_of(int blocks, int step) { return (blocks + step - 1) / step; }

// All threads of the CTA; ends with a barrier.
__device__ __forceinline__ void shared_geometry(SharedGeo* s, const DecodeArgs& a, int TQ, int step, int tid,
                                                int threads, bool report) {
  const int n = a.num_groups;
  const unsigned bad = load_groups(&s->g, a.group_start, a.prefix_blocks, n, a.B, a.mbps, tid, threads);
  if (bad && report && tid == 0) flag(a.err, bad);
  if (tid < 32) {
    int u = 0;
    long long x = 0;
    for (int base = 0; base < n; base += 32) {
      const int i = base + tid;
      int du = 0;
      long long dx = 0;
      if (i < n) {
        du = ((s->g.start[i + 1] - s->g.start[i]) * a.G + TQ - 1) / TQ * a.c.H;
        dx = (long long)du * steps_of(s->g.blocks[i], step);
      }
      int su = du;
      long long sx = dx;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int mu = __shfl_up_sync(kFull, su, o);
        const long long mx = __shfl_up_sync(kFull, sx, o);
        if (tid >= o) {
          su += mu;
          sx += mx;
        }
      }
      if (i < n) {
        s->unit0[i] = u + su - du;
        s->x0[i] = x + sx - dx;
      }
      u += __shfl_sync(kFull, su, 31);
      x += __shfl_sync(kFull, sx, 31);
    }
    if (tid == 0) {
      s->units = s->unit0[n] = u;
      s->T = s->x0[n] = x;
    }
  }
  __syncthreads();
}

// CTAs that share the range: never more than steps / kMinSteps, so that each owns some.
constexpr int kMinSteps = 4;
__device__ __forceinline__ int shared_ctas(const SharedGeo* s, int P) {
  const long long most = (s->T + kMinSteps - 1) / kMinSteps;
  return int(most < (long long)P ? most : (long long)P);
}

struct SharedUnit {
  int group, tile, h, u;
  long long start;  // its first step in the range
  int steps;
};

// The unit that holds step x < T.
__device__ __forceinline__ SharedUnit unit_at(const SharedGeo* s, int n, int H, int step, long long x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {  // the last group with x0 <= x: the earlier ones end before it
    const int mid = (lo + hi + 1) >> 1;
    if (s->x0[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  SharedUnit r;
  r.group = lo;
  r.steps = steps_of(s->g.blocks[lo], step);
  const int i = int((x - s->x0[lo]) / r.steps);
  r.tile = i / H;
  r.h = i % H;
  r.u = s->unit0[lo] + i;
  r.start = s->x0[lo] + (long long)i * r.steps;
  return r;
}

__device__ __forceinline__ void wait_for_suffix() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Tokens of the prefix that sequence b attends to.
__device__ __forceinline__ int prefix_len(const DecodeArgs& a, int b, int blocks) {
  const int L = min(max(__ldcg(a.seq_lens + b), 0), table_tokens(a.mbps, a.c.window));
  return min(max(L - a.c.window, 0), blocks * kBlock);
}

}  // namespace
}  // namespace kvq
