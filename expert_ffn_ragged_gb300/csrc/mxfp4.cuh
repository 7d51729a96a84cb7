// mxfp4.cuh -- the arithmetic of 4-bit microscaled blocks (32 elements, one E8M0 scale).
//
// The scale exponent is read off the bits of the block's largest magnitude: a biased exponent E
// stands for floor(log2 amax) = E - 127, and the scale is 2^(E - 127 - 2), kept as the byte
// max(E - 2, 0).  Dividing by it is a multiplication by an exact power of two, so the only
// rounding is the one to the eight E2M1 magnitudes (nearest even, above 6 to 6).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace rd {

constexpr int kMxBlock = 32;

// scale byte of a block from the bits of its largest magnitude (0xFF: a NaN or an infinity in it)
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 1 / scale; 0 for a block without finite values, whose codes are then 0
__device__ __forceinline__ float mx_inverse(uint32_t scale_byte) {
  return scale_byte == 255u ? 0.0f : __uint_as_float((254u - scale_byte) << 23);
}

// scale of a byte as f32 (2^-127 is a subnormal; 0xFF is NaN)
__device__ __forceinline__ float mx_scale(uint32_t scale_byte) {
  return scale_byte == 255u ? __uint_as_float(0x7FFFFFFFu)
                            : __uint_as_float(scale_byte == 0u ? 0x00400000u : scale_byte << 23);
}

// eight scaled values to eight codes, the first in the lowest four bits
__device__ __forceinline__ uint32_t mx_pack8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

}  // namespace rd
