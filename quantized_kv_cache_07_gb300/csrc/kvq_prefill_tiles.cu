// Chunked prefill on query tiles: the whole context (the kernel template lives in kvq_prefill_tiles.cuh).
#include "kvq_prefill_tiles.cuh"

namespace kvq {

bool prefill_tiles_supported(const CacheView& c) {
  const bool bits = ((c.k_bits == 8 || c.k_bits == 4) && (c.v_bits == 8 || c.v_bits == 4)) ||
                    (c.k_bits == 2 && c.v_bits == 2);
  return bits && (c.q_bits == 0 || c.q_bits == 16 || c.q_bits == 8 || c.q_bits == 32) && c.window == 0;
}

cudaError_t launch_prefill_tiles(const DecodeArgs& a, cudaStream_t s) {
  const bool loq = a.c.q_bits == 32;
  if (a.c.asym) return loq ? launch_tiles<true, true, false>(a, s) : launch_tiles<true, false, false>(a, s);
  return loq ? launch_tiles<false, true, false>(a, s) : launch_tiles<false, false, false>(a, s);
}

}  // namespace kvq
