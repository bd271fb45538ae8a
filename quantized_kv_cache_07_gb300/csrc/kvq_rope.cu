// Rotary positions with the cache write (kvq_rope.cuh) and their table.
#include "kvq_rope.cuh"

namespace kvq {
namespace {

__global__ void __launch_bounds__(256) rope_table_kernel(const RopeFreqs f, int pairs, long long n, float* table) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  double s, c;
  sincos(double(i / pairs) * f.f[i % pairs], &s, &c);
  reinterpret_cast<float2*>(table)[i] = make_float2(float(f.amplitude * c), float(f.amplitude * s));
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t s) { return launch_rope<false>(a, s); }

cudaError_t launch_rope_table(const RopeFreqs& f, int pairs, int max_pos, float* table, cudaStream_t s) {
  const long long n = (long long)max_pos * pairs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((n + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, rope_table_kernel, f, pairs, n, table);
}

}  // namespace kvq
