// Suffix kernels of kvq_decode_shared (kvq_suffix.cuh) in the two-part mode (q_bits 32).
#include "kvq_suffix.cuh"

namespace kvq {

int suffix_ctas_q32(const CacheView& c, int B) {
  return suffix_by_format<true>(c, [&](auto k) { return decltype(k)::ctas(B); });
}

cudaError_t launch_suffix_q32(const SharedArgs& a, cudaStream_t s) {
  return suffix_by_format<true>(a.d.c, [&](auto k) { return decltype(k)::launch(a, s); });
}

}  // namespace kvq
