// mxfp4.cu -- rows to 4-bit microscaled blocks and back, and the layout of 4-bit expert weights.
//
// HBM streams: quantisation reads 2 bytes an element and writes 17/32 (times topk when the rows go
// to their packed places at once), dequantisation the other way round.
#include <cuda_runtime.h>
#include <stdint.h>

#include "glu_math.cuh"
#include "moe_args.h"
#include "mxfp4.cuh"

namespace rd {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantWarps = kQuantThreads / 32;

__device__ __forceinline__ int32_t rows_below(const int32_t* limit, int32_t rows) {
  if (limit == nullptr) return rows;
  const int32_t v = *limit;
  return v < 0 ? 0 : (v > rows ? rows : v);
}

// largest magnitude bits of eight packed bf16 values, as f32 bits
__device__ __forceinline__ uint32_t amax8(uint4 v) {
  const uint32_t c[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(c[i] << 16, c[i] & 0xFFFF0000u));
  return m;
}

__device__ __forceinline__ uint32_t pack_scaled(uint4 v, float inv) {
  const float f[8] = {bf16_lo(v.x) * inv, bf16_hi(v.x) * inv, bf16_lo(v.y) * inv, bf16_hi(v.y) * inv,
                      bf16_lo(v.z) * inv, bf16_hi(v.z) * inv, bf16_lo(v.w) * inv, bf16_hi(v.w) * inv};
  return mx_pack8(f);
}

// A warp takes 256 elements of a row: lane i eight of them, four lanes a block.
__global__ void __launch_bounds__(kQuantThreads) mxfp4_quantize_kernel(const QuantArgs a) {
  const int lane = threadIdx.x & 31;
  const int32_t L = rows_below(a.limit, a.rows);
  const int pieces = (a.k + 255) / 256;
  const int64_t units = static_cast<int64_t>(L) * pieces;
  const uint4* x = static_cast<const uint4*>(a.x);
  const int vecs = a.k / 8, blocks = a.k / kMxBlock;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kQuantWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kQuantWarps) {
    const int64_t r = u / pieces;
    const int piece = static_cast<int>(u - r * pieces);
    const int v = piece * 32 + lane;
    uint4 xv = make_uint4(0, 0, 0, 0);
    if (v < vecs) xv = x[r * vecs + v];
    uint32_t m = amax8(xv);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const uint32_t sb = mx_scale_byte(m);
    uint32_t codes = pack_scaled(xv, mx_inverse(sb));
    if (sb == 255u) codes = 0;  // inf * 0 is NaN: the codes of such a block are 0
    const int block = piece * 8 + (lane >> 2);
    auto put = [&](int64_t row) {
      if (v < vecs) reinterpret_cast<uint32_t*>(a.q + row * (a.k / 2))[v] = codes;
      uint8_t* s = a.scales + row * a.scale_width;
      if ((lane & 3) == 0 && block < blocks) s[block] = static_cast<uint8_t>(sb);
      if (piece == pieces - 1 && blocks + lane < a.scale_width) s[blocks + lane] = 0;
    };
    if (a.pos == nullptr) {
      put(r);
    } else {
      for (int k = 0; k < a.topk; ++k) {
        const int32_t p = a.pos[r * a.topk + k];
        if (p >= 0 && p < a.out_rows) put(p);
      }
    }
  }
}

__global__ void __launch_bounds__(kQuantThreads)
    mxfp4_dequantize_kernel(const QuantArgs a, uint4* __restrict__ out) {
  const int32_t L = rows_below(a.limit, a.rows);
  const int vecs = a.k / 8;
  const int64_t units = static_cast<int64_t>(L) * vecs;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kQuantThreads + threadIdx.x; u < units;
       u += static_cast<int64_t>(gridDim.x) * kQuantThreads) {
    const int64_t r = u / vecs;
    const int v = static_cast<int>(u - r * vecs);
    const uint32_t c = reinterpret_cast<const uint32_t*>(a.q)[u];
    const float s = mx_scale(a.scales[r * a.scale_width + v / 4]);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = mx_code_value(c >> (4 * i)) * s;
    out[u] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                        pack_bf16x2(f[6], f[7]));
  }
}

// Weights [g, k, n] to rows along k: a thread owns one output column n and one block of 32 k.
// Reads are coalesced over n; each thread writes its 16 bytes of codes.
__global__ void __launch_bounds__(kQuantThreads)
    mxfp4_weights_kernel(const __nv_bfloat16* __restrict__ rhs, uint8_t* __restrict__ q,
                         uint8_t* __restrict__ scales, int32_t k, int32_t n, int32_t scale_width) {
  const int col = blockIdx.x * kQuantThreads + threadIdx.x;
  const int block = blockIdx.y;
  const int64_t e = blockIdx.z;
  if (col >= n) return;
  uint8_t* s = scales + (e * n + col) * scale_width + block;
  if (block >= k / kMxBlock) {
    *s = 0;
    return;
  }
  const __nv_bfloat16* src = rhs + (e * k + static_cast<int64_t>(block) * kMxBlock) * n + col;
  float v[kMxBlock];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i) {
    v[i] = __bfloat162float(src[static_cast<int64_t>(i) * n]);
    m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
  const uint32_t sb = mx_scale_byte(m);
  const float inv = mx_inverse(sb);
  uint32_t codes[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v[8 * j + i] * inv;
    codes[j] = sb == 255u ? 0u : mx_pack8(f);
  }
  *reinterpret_cast<uint4*>(q + (e * n + col) * (k / 2) + block * 16) =
      make_uint4(codes[0], codes[1], codes[2], codes[3]);
  *s = static_cast<uint8_t>(sb);
}

int quant_grid(int64_t blocks, int sms) {
  return static_cast<int>(blocks < 8 * static_cast<int64_t>(sms) ? blocks : 8 * static_cast<int64_t>(sms));
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const QuantArgs& a, int sms, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(a.rows) * ((a.k + 255) / 256);
  mxfp4_quantize_kernel<<<quant_grid((units + kQuantWarps - 1) / kQuantWarps, sms), kQuantThreads, 0,
                          stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequantize(const QuantArgs& a, void* out, int sms, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(a.rows) * (a.k / 8);
  mxfp4_dequantize_kernel<<<quant_grid((units + kQuantThreads - 1) / kQuantThreads, sms),
                            kQuantThreads, 0, stream>>>(a, static_cast<uint4*>(out));
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_quantize_weights(const void* rhs, uint8_t* q, uint8_t* scales, int32_t g,
                                          int32_t k, int32_t n, int32_t scale_width,
                                          cudaStream_t stream) {
  const dim3 grid((n + kQuantThreads - 1) / kQuantThreads, scale_width, g);
  mxfp4_weights_kernel<<<grid, kQuantThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(rhs), q,
                                                           scales, k, n, scale_width);
  return cudaGetLastError();
}

}  // namespace rd
