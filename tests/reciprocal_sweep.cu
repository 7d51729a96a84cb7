// The router's reciprocal against the correctly rounded one, for every float of its range
// (tests/test_gpu_route_exact.py builds and runs it).
#include <cuda_runtime.h>
#include <stdint.h>

#include "route_math.cuh"

namespace {

__global__ void sweep(uint32_t first, uint32_t count, unsigned long long* wrong, unsigned int* lowest) {
  const uint32_t stride = gridDim.x * blockDim.x;
  for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < count; i += stride) {
    const float d = __uint_as_float(first + i);
    if (__float_as_uint(rd::reciprocal_fast(d)) != __float_as_uint(__frcp_rn(d))) {
      atomicAdd(wrong, 1ull);
      atomicMin(lowest, first + i);
    }
  }
}

}  // namespace

// Floats in [1, kFastRcp): how many there are, how many reciprocals differ, and the lowest such float's
// bits.  Returns a CUDA error code.
extern "C" int reciprocal_sweep(unsigned int* count, unsigned long long* wrong, unsigned int* lowest) {
  const float lo = 1.0f, hi = rd::kFastRcp;
  uint32_t first, last;
  __builtin_memcpy(&first, &lo, 4);
  __builtin_memcpy(&last, &hi, 4);
  *count = last - first;
  unsigned long long* w;
  unsigned int* l;
  cudaError_t e = cudaMalloc(&w, sizeof(*w));
  if (e == cudaSuccess) e = cudaMalloc(&l, sizeof(*l));
  if (e == cudaSuccess) e = cudaMemset(w, 0, sizeof(*w));
  if (e == cudaSuccess) e = cudaMemset(l, 0xFF, sizeof(*l));
  if (e == cudaSuccess) {
    sweep<<<1216, 256>>>(first, last - first, w, l);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaMemcpy(wrong, w, sizeof(*w), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemcpy(lowest, l, sizeof(*l), cudaMemcpyDeviceToHost);
  cudaFree(w);
  cudaFree(l);
  return static_cast<int>(e);
}
