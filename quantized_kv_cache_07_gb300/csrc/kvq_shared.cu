// The merge of kvq_decode_shared: each query's prefix and suffix records, by log-sum-exp.
//
// One warp per query vector; lane l holds dims 4l..4l+3.  The vector's unit and the
// CTAs that own its steps follow from the same arithmetic as in the prefix
// kernel, so nothing is counted and no order depends on the scheduling.
#include "kvq_shared.cuh"

namespace kvq {
namespace {

constexpr int kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads) shared_merge_kernel(const SharedArgs sa, int step) {
  __shared__ SharedGeo geo;
  const DecodeArgs& a = sa.d;
  const int tid = threadIdx.x, lane = tid & 31;
  // the groups are as old as what the prefix kernel reads before its wait
  shared_geometry(&geo, a, sa.sl.unit, step, tid, kMergeThreads, false);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long q = (long long)blockIdx.x * (kMergeThreads / 32) + (tid >> 5);
  const bool any = q < (long long)a.B * a.Hq;
  const int b = any ? int(q / a.Hq) : 0, hq = any ? int(q % a.Hq) : 0, h = hq / a.G, hj = hq % a.G;
  // ---- where the records are: prefix ones (np), the suffix's chunks (ns), the window's
  const int2 ch = reinterpret_cast<const int2*>(a.ws + sa.sl.off_chunks)[b];
  const int2 last = reinterpret_cast<const int2*>(a.ws + sa.sl.off_chunks)[a.B - 1];
  if (!any) return;
  const int H = a.c.H, ns = ch.y;
  const size_t first_s = size_t(ch.x) + size_t(h) * ns;  // suffix record of chunk 0 of this unit
  const size_t win = size_t(last.x) + size_t(last.y) * H + size_t(b) * H + h;
  int np = 0, two = 0, v = 0;
  size_t first_p = 0;
  const int g = group_of(&geo.g, a.num_groups, b);
  if (g >= 0 && geo.g.blocks[g] > 0) {
    v = (b - geo.g.start[g]) * a.G + hj;
    const int tile = v / sa.sl.unit, steps = steps_of(geo.g.blocks[g], step);
    const int i = tile * H + h, u = geo.unit0[g] + i;
    const long long x = geo.x0[g] + (long long)i * steps;
    const int Pe = shared_ctas(&geo, sa.sl.ctas);
    const long long c0 = cta_of(x, geo.T, Pe), c1 = cta_of(x + steps - 1, geo.T, Pe);
    // On tcgen05 a unit of at most 128 vectors has two records per CTA, the second one's rows behind the first's.
    const int nv = min((geo.g.start[g + 1] - geo.g.start[g]) * a.G - tile * sa.sl.unit, sa.sl.unit);
    two = sa.sl.tc && nv <= sa.sl.tile / 2 ? 1 : 0;
    np = int(c1 - c0 + 1) << two;
    first_p = size_t(c0 + u) * sa.sl.tile + v % sa.sl.unit;
  }
  const float* pm = reinterpret_cast<const float*>(a.ws + sa.sl.off_m);
  const float* pl = reinterpret_cast<const float*>(a.ws + sa.sl.off_l);
  const float4* po = reinterpret_cast<const float4*>(a.ws + sa.sl.off_rec);
  const float* sm = reinterpret_cast<const float*>(a.ws + sa.sl.off_sm);
  const float* sl = reinterpret_cast<const float*>(a.ws + sa.sl.off_sl);
  const float4* so = reinterpret_cast<const float4*>(a.ws + sa.sl.off_so);
  const int n = np + ns + (a.c.window > 0 ? 1 : 0);
  float M = kNegInf, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kR = 8;  // records in flight
  for (int i0 = 0; i0 < n; i0 += kR) {
    float mr[kR], lr[kR];
    float4 orr[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int i = i0 + r;
      mr[r] = kNegInf;
      lr[r] = 0.f;
      orr[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < np) {
        const size_t at = first_p + size_t(i >> two) * sa.sl.tile + (two && (i & 1) ? sa.sl.tile / 2 : 0);
        mr[r] = pm[at];
        lr[r] = pl[at];
        orr[r] = po[at * (kHeadDim / 4) + lane];
      } else if (i < n) {
        const size_t at = (i < np + ns ? first_s + (i - np) : win) * a.G + hj;
        mr[r] = sm[at];
        lr[r] = sl[at];
        orr[r] = so[at * (kHeadDim / 4) + lane];
      }
      if (mr[r] == kNegInf) orr[r] = make_float4(0.f, 0.f, 0.f, 0.f);  // a record without a token may hold anything
    }
    float Mn = M;
#pragma unroll
    for (int r = 0; r < kR; ++r) Mn = fmaxf(Mn, mr[r]);
    const float rs = M == kNegInf ? 0.f : exp2f(M - Mn);
    l *= rs;
    o.x *= rs;
    o.y *= rs;
    o.z *= rs;
    o.w *= rs;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const float w = mr[r] == kNegInf ? 0.f : exp2f(mr[r] - Mn);
      l = fmaf(w, lr[r], l);
      o.x = fmaf(w, orr[r].x, o.x);
      o.y = fmaf(w, orr[r].y, o.y);
      o.z = fmaf(w, orr[r].z, o.z);
      o.w = fmaf(w, orr[r].w, o.w);
    }
    M = Mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;  // nothing attended: out = 0
  if (a.out_fp32) {
    reinterpret_cast<float4*>(a.out)[q * (kHeadDim / 4) + lane] =
        make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  } else {
    reinterpret_cast<uint2*>(a.out)[q * (kHeadDim / 4) + lane] =
        make_uint2(pack_bf162(o.x * inv, o.y * inv), pack_bf162(o.z * inv, o.w * inv));
  }
  if (lane == 0 && a.lse) a.lse[q] = l > 0.f ? (M + log2f(l)) * kLn2 : kNegInf;
}

}  // namespace

cudaError_t launch_shared_merge(const SharedArgs& a, cudaStream_t s) {
  const long long warps = (long long)a.d.B * a.d.Hq;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((warps + kMergeThreads / 32 - 1) / (kMergeThreads / 32)));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_merge_kernel, a, kConsumerWarps);
}

}  // namespace kvq
