// Chunked prefill with sinks on tcgen05 (kvq_sinks_tc.cuh): a cluster a unit.
#include "kvq_sinks_tc.cuh"

namespace kvq {

cudaError_t sinks_tc_clusters(const CacheView& v, int ctas, int c, int* n) {
  return by_format<true>(v, [&](auto k) {
    const cudaError_t e = k.prepare();
    return e != cudaSuccess ? e : k.clusters(ctas, c, n);
  });
}

cudaError_t launch_sinks_tc_shared(const DecodeArgs& a, int units, int rows, int c, cudaStream_t s) {
  return by_format<true>(a.c, [&](auto k) {
    const cudaError_t e = k.prepare();
    return e != cudaSuccess ? e : k.launch(a, units, rows, units << c, c, s);
  });
}

}  // namespace kvq
