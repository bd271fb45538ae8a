// Norms of the heads and rotary positions with the cache write (kvq_rope.cuh).
#include "kvq_rope.cuh"

namespace kvq {

cudaError_t launch_norm_rope_append(const RopeArgs& a, cudaStream_t s) { return launch_rope<true>(a, s); }

}  // namespace kvq
