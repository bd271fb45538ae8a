// Attention with sinks and a sliding window, one decode step or the split rows of a chunk: the decode kernel
// (kvq_decode_impl.cuh, SPAN) over the blocks that are seen, with its masks at the sinks' end and the
// window's start.  Symmetric formats and bf16 blocks; kvq_sinks_asym.cu and kvq_sinks_q32.cu hold the others.
#include "kvq_decode_impl.cuh"

namespace kvq {

int sinks_ctas_per_sm(const CacheView& c, int B, bool rows) {
  const int kb = c.k_bits, vb = c.v_bits;
  if (c.q_bits == 32 && kb != 16) return sinks_ctas_per_sm_q32(c, B, rows);
  if (c.asym) return sinks_ctas_per_sm_asym(c, B, rows);
  if (kb == 8 && vb == 8) return Kernel<8, 8, false, false, true>::ctas_per_sm(B, rows);
  if (kb == 4 && vb == 4) return Kernel<4, 4, false, false, true>::ctas_per_sm(B, rows);
  if (kb == 4 && vb == 8) return Kernel<4, 8, false, false, true>::ctas_per_sm(B, rows);
  if (kb == 8 && vb == 4) return Kernel<8, 4, false, false, true>::ctas_per_sm(B, rows);
  if (kb == 2 && vb == 2) return Kernel<2, 2, false, false, true>::ctas_per_sm(B, rows);
  if (kb == 16 && vb == 16) return Kernel<16, 16, false, false, true>::ctas_per_sm(B, rows);
  return 0;
}

cudaError_t launch_sinks(const DecodeArgs& a, cudaStream_t s) {
  const int kb = a.c.k_bits, vb = a.c.v_bits;
  if (a.c.q_bits == 32 && kb != 16) return launch_sinks_q32(a, s);
  if (a.c.asym) return launch_sinks_asym(a, s);
  if (kb == 8 && vb == 8) return Kernel<8, 8, false, false, true>::launch(a, s);
  if (kb == 4 && vb == 4) return Kernel<4, 4, false, false, true>::launch(a, s);
  if (kb == 4 && vb == 8) return Kernel<4, 8, false, false, true>::launch(a, s);
  if (kb == 8 && vb == 4) return Kernel<8, 4, false, false, true>::launch(a, s);
  if (kb == 2 && vb == 2) return Kernel<2, 2, false, false, true>::launch(a, s);
  if (kb == 16 && vb == 16) return Kernel<16, 16, false, false, true>::launch(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
