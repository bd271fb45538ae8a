// Attention with sinks and a sliding window, query and value weights in two fp16 parts (q_bits 32, and under a key
// factor).
#include "kvq_decode_impl.cuh"

namespace kvq {

int sinks_ctas_per_sm_q32(const CacheView& c, int B, bool rows) {
  const int kb = c.k_bits, vb = c.v_bits;
  if (c.asym) {
    if (kb == 8 && vb == 8) return Kernel<8, 8, true, true, true>::ctas_per_sm(B, rows);
    if (kb == 4 && vb == 4) return Kernel<4, 4, true, true, true>::ctas_per_sm(B, rows);
    if (kb == 4 && vb == 8) return Kernel<4, 8, true, true, true>::ctas_per_sm(B, rows);
    if (kb == 8 && vb == 4) return Kernel<8, 4, true, true, true>::ctas_per_sm(B, rows);
    if (kb == 2 && vb == 2) return Kernel<2, 2, true, true, true>::ctas_per_sm(B, rows);
    return 0;
  }
  if (kb == 8 && vb == 8) return Kernel<8, 8, false, true, true>::ctas_per_sm(B, rows);
  if (kb == 4 && vb == 4) return Kernel<4, 4, false, true, true>::ctas_per_sm(B, rows);
  if (kb == 4 && vb == 8) return Kernel<4, 8, false, true, true>::ctas_per_sm(B, rows);
  if (kb == 8 && vb == 4) return Kernel<8, 4, false, true, true>::ctas_per_sm(B, rows);
  if (kb == 2 && vb == 2) return Kernel<2, 2, false, true, true>::ctas_per_sm(B, rows);
  return 0;
}

cudaError_t launch_sinks_q32(const DecodeArgs& a, cudaStream_t s) {
  const int kb = a.c.k_bits, vb = a.c.v_bits;
  if (a.c.asym) {
    if (kb == 8 && vb == 8) return Kernel<8, 8, true, true, true>::launch(a, s);
    if (kb == 4 && vb == 4) return Kernel<4, 4, true, true, true>::launch(a, s);
    if (kb == 4 && vb == 8) return Kernel<4, 8, true, true, true>::launch(a, s);
    if (kb == 8 && vb == 4) return Kernel<8, 4, true, true, true>::launch(a, s);
    if (kb == 2 && vb == 2) return Kernel<2, 2, true, true, true>::launch(a, s);
    return cudaErrorInvalidValue;
  }
  if (kb == 8 && vb == 8) return Kernel<8, 8, false, true, true>::launch(a, s);
  if (kb == 4 && vb == 4) return Kernel<4, 4, false, true, true>::launch(a, s);
  if (kb == 4 && vb == 8) return Kernel<4, 8, false, true, true>::launch(a, s);
  if (kb == 8 && vb == 4) return Kernel<8, 4, false, true, true>::launch(a, s);
  if (kb == 2 && vb == 2) return Kernel<2, 2, false, true, true>::launch(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
