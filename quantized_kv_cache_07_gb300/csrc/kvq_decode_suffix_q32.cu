// Suffix decode kernels (kvq_decode_suffix.cu) of the two-part mode (q_bits 32).
#include "kvq_decode_impl.cuh"

namespace kvq {

namespace {
template <class F>
auto by_format(int kb, int vb, bool asym, F f) {
  if (kb == 8 && vb == 8) return asym ? f(Kernel<8, 8, true, true, true>{}) : f(Kernel<8, 8, false, true, true>{});
  if (kb == 4 && vb == 4) return asym ? f(Kernel<4, 4, true, true, true>{}) : f(Kernel<4, 4, false, true, true>{});
  if (kb == 4 && vb == 8) return asym ? f(Kernel<4, 8, true, true, true>{}) : f(Kernel<4, 8, false, true, true>{});
  if (kb == 8 && vb == 4) return asym ? f(Kernel<8, 4, true, true, true>{}) : f(Kernel<8, 4, false, true, true>{});
  return asym ? f(Kernel<2, 2, true, true, true>{}) : f(Kernel<2, 2, false, true, true>{});
}
}  // namespace

int suffix_ctas_per_sm_q32(int k_bits, int v_bits, bool asym, int B) {
  return by_format(k_bits, v_bits, asym, [&](auto k) { return decltype(k)::ctas_per_sm(B, true); });
}

cudaError_t launch_suffix_q32(const DecodeArgs& a, cudaStream_t s) {
  return by_format(a.c.k_bits, a.c.v_bits, a.c.asym != 0, [&](auto k) { return decltype(k)::launch(a, s); });
}

}  // namespace kvq
