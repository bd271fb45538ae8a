// Chunked prefill on query tiles with sinks and a sliding window (the kernel template lives in kvq_prefill_tiles.cuh).
#include "kvq_prefill_tiles.cuh"

namespace kvq {

cudaError_t launch_sinks_tiles(const DecodeArgs& a, cudaStream_t s) {
  const bool loq = a.c.q_bits == 32;
  if (a.c.asym) return loq ? launch_tiles<true, true, true>(a, s) : launch_tiles<true, false, true>(a, s);
  return loq ? launch_tiles<false, true, true>(a, s) : launch_tiles<false, false, true>(a, s);
}

}  // namespace kvq
