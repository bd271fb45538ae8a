// Suffix kernels of kvq_decode_shared (kvq_suffix.cuh), one-part query modes and bf16 blocks.
#include "kvq_suffix.cuh"

namespace kvq {

int suffix_ctas(const CacheView& c, int B) {
  if (c.q_bits == 32 && c.k_bits != 16) return suffix_ctas_q32(c, B);
  return suffix_by_format<false>(c, [&](auto k) { return decltype(k)::ctas(B); });
}

cudaError_t launch_suffix(const SharedArgs& a, cudaStream_t s) {
  if (a.d.c.q_bits == 32 && a.d.c.k_bits != 16) return launch_suffix_q32(a, s);
  return suffix_by_format<false>(a.d.c, [&](auto k) { return decltype(k)::launch(a, s); });
}

}  // namespace kvq
