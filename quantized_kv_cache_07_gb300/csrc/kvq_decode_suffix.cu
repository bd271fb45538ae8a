// Decode kernels over the tokens behind a shared prefix (kvq_decode_shared):
// the decode kernel with the block table read from each sequence's first own
// block, one-part query modes.  The two-part mode is in kvq_decode_suffix_q32.cu.
#include "kvq_decode_impl.cuh"

namespace kvq {

namespace {
template <class F>
auto by_format(int kb, int vb, bool asym, F f) {
  if (kb == 8 && vb == 8) return asym ? f(Kernel<8, 8, true, false, true>{}) : f(Kernel<8, 8, false, false, true>{});
  if (kb == 4 && vb == 4) return asym ? f(Kernel<4, 4, true, false, true>{}) : f(Kernel<4, 4, false, false, true>{});
  if (kb == 4 && vb == 8) return asym ? f(Kernel<4, 8, true, false, true>{}) : f(Kernel<4, 8, false, false, true>{});
  if (kb == 8 && vb == 4) return asym ? f(Kernel<8, 4, true, false, true>{}) : f(Kernel<8, 4, false, false, true>{});
  if (kb == 2 && vb == 2) return asym ? f(Kernel<2, 2, true, false, true>{}) : f(Kernel<2, 2, false, false, true>{});
  return f(Kernel<16, 16, false, false, true>{});
}
}  // namespace

int suffix_ctas_per_sm_for(int k_bits, int v_bits, bool asym, int q_bits, int B) {
  if (q_bits == 32 && k_bits != 16) return suffix_ctas_per_sm_q32(k_bits, v_bits, asym, B);
  return by_format(k_bits, v_bits, asym, [&](auto k) { return decltype(k)::ctas_per_sm(B, true); });
}

cudaError_t launch_suffix(const DecodeArgs& a, cudaStream_t s) {
  if (a.c.q_bits == 32 && a.c.k_bits != 16) return launch_suffix_q32(a, s);
  return by_format(a.c.k_bits, a.c.v_bits, a.c.asym != 0, [&](auto k) { return decltype(k)::launch(a, s); });
}

}  // namespace kvq
