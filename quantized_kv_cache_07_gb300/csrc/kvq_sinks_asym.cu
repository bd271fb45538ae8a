// Attention with sinks and a sliding window against asymmetric blocks (scale and zero point).
#include "kvq_decode_impl.cuh"

namespace kvq {

int sinks_ctas_per_sm_asym(const CacheView& c, int B, bool rows) {
  const int kb = c.k_bits, vb = c.v_bits;
  if (kb == 8 && vb == 8) return Kernel<8, 8, true, false, true>::ctas_per_sm(B, rows);
  if (kb == 4 && vb == 4) return Kernel<4, 4, true, false, true>::ctas_per_sm(B, rows);
  if (kb == 4 && vb == 8) return Kernel<4, 8, true, false, true>::ctas_per_sm(B, rows);
  if (kb == 8 && vb == 4) return Kernel<8, 4, true, false, true>::ctas_per_sm(B, rows);
  if (kb == 2 && vb == 2) return Kernel<2, 2, true, false, true>::ctas_per_sm(B, rows);
  return 0;
}

cudaError_t launch_sinks_asym(const DecodeArgs& a, cudaStream_t s) {
  const int kb = a.c.k_bits, vb = a.c.v_bits;
  if (kb == 8 && vb == 8) return Kernel<8, 8, true, false, true>::launch(a, s);
  if (kb == 4 && vb == 4) return Kernel<4, 4, true, false, true>::launch(a, s);
  if (kb == 4 && vb == 8) return Kernel<4, 8, true, false, true>::launch(a, s);
  if (kb == 8 && vb == 4) return Kernel<8, 4, true, false, true>::launch(a, s);
  if (kb == 2 && vb == 2) return Kernel<2, 2, true, false, true>::launch(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
