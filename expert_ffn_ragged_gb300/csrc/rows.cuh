// rows.cuh -- what the row kernels of rd_block.h share: eight elements of a row as f32, the row
// limit, and sums across the threads of a row.
//
// A thread moves eight elements at a time: 16 bytes of bf16 or 32 of f32, each one load or store
// (the f32 form needs a 32-byte boundary).  Two 16-byte accesses 32 bytes apart would touch every
// sector of a warp's rows twice.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "glu_math.cuh"

namespace rd {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ int32_t rows_within(const int32_t* limit, int32_t rows) {
  if (limit == nullptr) return rows;
  const int32_t v = *limit;
  return v < 0 ? 0 : (v > rows ? rows : v);
}

// eight elements as they lie in memory
template <class E>
struct Raw8;
template <>
struct Raw8<bf16> {
  uint32_t w[4];
};
template <>
struct Raw8<float> {
  uint32_t w[8];
};

__device__ __forceinline__ void load_raw(Raw8<bf16>& r, const bf16* p) {
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
               : "l"(p)
               : "memory");
}

__device__ __forceinline__ void load_raw(Raw8<float>& r, const float* p) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]),
                 "=r"(r.w[6]), "=r"(r.w[7])
               : "l"(p)
               : "memory");
}

__device__ __forceinline__ void widen(const Raw8<bf16>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(r.w[i]);
    v[2 * i + 1] = bf16_hi(r.w[i]);
  }
}

__device__ __forceinline__ void widen(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
}

template <class E>
__device__ __forceinline__ void load8(const E* p, float (&v)[8]) {
  Raw8<E> r;
  load_raw(r, p);
  widen(r, v);
}

__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// eight f32 of a weight or bias, from a 16-byte boundary (reused from row to row: through L1)
__device__ __forceinline__ void load8_param(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// ---- quads: four elements, the unit that a thread copies to shared memory ahead of its use (16 bytes
// of f32, 8 of bf16: a warp's copies are whole lines in both)
template <class E>
struct Quad;
template <>
struct Quad<float> {
  using Raw = float4;
};
template <>
struct Quad<bf16> {
  using Raw = uint2;
};

__device__ __forceinline__ void quad_copy(float4* dst, const float* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void quad_copy(uint2* dst, const bf16* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the N newest groups of this thread's copies have landed
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void widen(float4 r, float2 (&v)[2]) {
  v[0] = make_float2(r.x, r.y);
  v[1] = make_float2(r.z, r.w);
}
__device__ __forceinline__ void widen(uint2 r, float2 (&v)[2]) {
  v[0] = make_float2(bf16_lo(r.x), bf16_hi(r.x));
  v[1] = make_float2(bf16_lo(r.y), bf16_hi(r.y));
}
__device__ __forceinline__ void store4(float* p, const float2 (&v)[2]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
}
__device__ __forceinline__ void store4(bf16* p, const float2 (&v)[2]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
}

// N sums over the T threads of a row (T = 32: a warp; else the whole block), in a fixed order, the same
// in every thread, with one barrier.  The words of `slot` [T / 32][N] may be written again only after the
// barrier of another call in between.
template <int T, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* slot) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
  if (T == 32) return;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) slot[(threadIdx.x >> 5) * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const float4 p = reinterpret_cast<const float4*>(slot)[w * (N / 4) + i];
        v[4 * i] += p.x, v[4 * i + 1] += p.y, v[4 * i + 2] += p.z, v[4 * i + 3] += p.w;
      }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float2 p = reinterpret_cast<const float2*>(slot)[w * (N / 2) + i];
        v[2 * i] += p.x, v[2 * i + 1] += p.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += slot[w * N + i];
    }
  }
}

}  // namespace rd
