// route_math.cuh -- the reciprocal of the router's scores.
#pragma once

#include <cuda_runtime.h>

namespace rd {

// The correctly rounded 1 / d for d in [1, kFastRcp): the hardware approximation and one Newton step
// with fused multiply-adds, r + r (1 - d r), which rounds correctly when r is within an ulp
// (P. Markstein, IA-64 and Elementary Functions, 2000, for all mantissas but the one of all ones);
// tests/reciprocal_sweep.cu compares it with the correctly rounded reciprocal for every float in the range.
constexpr float kFastRcp = 1.0e37f;
__device__ __forceinline__ float reciprocal_fast(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return __fmaf_rn(r, __fmaf_rn(-d, r, 1.0f), r);
}

}  // namespace rd
