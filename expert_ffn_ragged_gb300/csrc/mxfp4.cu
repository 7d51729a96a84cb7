// mxfp4.cu -- rows to 4-bit microscaled blocks and back, and the layout of 4-bit expert weights.
//
// HBM streams: quantisation reads 2 bytes an element and writes 17/32 (times topk when the rows go
// to their packed places at once), dequantisation the other way round.  16381 rows of 4096 take 27 us one
// way (170 MB: 6.3 TB/s) and 27 us the other; 28160 rows to eight packed rows each 112.5 us (721 MB: 6.4
// TB/s); the issue slots are 64 % busy, so the arithmetic stays packed: maxima of two bf16 halves at once,
// and the scaling in bf16, where a power of two is exact.  Weights, once a model: 128 x 4096 x 1536 550 us
// (2.05 GB: 3.7 TB/s), bound by their stores of 16 bytes in rows k / 2 apart.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "glu_math.cuh"
#include "launch.h"
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
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                              __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  return max(m << 16, m & 0xFFFF0000u);
}

// Eight bf16 values times an exact power of two (a bf16 number too), in bf16: exact, except that
// values far below the smallest level may become 0, which they round to.
__device__ __forceinline__ uint32_t pack_scaled(uint4 v, float inv) {
  const __nv_bfloat162 f2 = __float2bfloat162_rn(inv);
  const uint32_t c[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&c[i]), f2);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&p);
    f[2 * i] = bf16_lo(u);
    f[2 * i + 1] = bf16_hi(u);
  }
  return mx_pack8(f);
}

constexpr int kQuantBatch = 4;  // pieces of 256 elements of a row that a warp has in flight

// A warp takes up to four pieces of 256 elements of a row: lane i eight of each, four lanes a block.
template <bool SEND>
__global__ void __launch_bounds__(kQuantThreads) mxfp4_quantize_kernel(const QuantArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int32_t L = rows_below(a.limit, a.rows);
  const int vecs = a.k / 8, blocks = a.k / kMxBlock;
  const unsigned runs = (vecs + 32 * kQuantBatch - 1) / (32 * kQuantBatch);  // of four pieces, a row
  const int64_t units = static_cast<int64_t>(L) * runs;
  const uint4* x = static_cast<const uint4*>(a.x);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kQuantWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kQuantWarps) {
    const int64_t r = units <= 0xFFFFFFFFll ? static_cast<unsigned>(u) / runs : u / runs;
    const int run = static_cast<int>(u - r * runs);
    const int v0 = run * 32 * kQuantBatch + lane;
    uint4 xv[kQuantBatch];
    uint32_t codes[kQuantBatch], sb[kQuantBatch];
#pragma unroll
    for (int b = 0; b < kQuantBatch; ++b) {
      xv[b] = make_uint4(0, 0, 0, 0);
      if (v0 + 32 * b < vecs) xv[b] = x[r * vecs + v0 + 32 * b];
    }
    const int32_t p_lane = SEND && lane < a.topk ? a.pos[r * a.topk + lane] : -1;
#pragma unroll
    for (int b = 0; b < kQuantBatch; ++b) {
      uint32_t m = amax8(xv[b]);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      sb[b] = mx_scale_byte(m);
      codes[b] = sb[b] == 255u ? 0u : pack_scaled(xv[b], mx_inverse(sb[b]));  // inf * 0 is NaN
    }
    auto put = [&](int64_t row) {
      uint32_t* q = reinterpret_cast<uint32_t*>(a.q + row * (a.k / 2));
      uint8_t* s = a.scales + row * a.scale_width;
#pragma unroll
      for (int b = 0; b < kQuantBatch; ++b) {
        const int v = v0 + 32 * b;
        if (v < vecs) {
          q[v] = codes[b];
          if ((lane & 3) == 0) s[v >> 2] = static_cast<uint8_t>(sb[b]);
        }
      }
      if (run == static_cast<int>(runs) - 1 && blocks + lane < a.scale_width) s[blocks + lane] = 0;
    };
    if (!SEND) {
      put(r);
    } else {
      for (int k = 0; k < a.topk; ++k) {
        const int32_t p = __shfl_sync(0xFFFFFFFFu, p_lane, k);
        if (p >= 0 && p < a.out_rows) put(p);
      }
    }
  }
}

// two values of a byte of codes
__device__ __forceinline__ float2 code_pair(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 lo, hi;\n\t"
      "mov.b16 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, lo;\n\t}"
      : "=r"(h)
      : "h"(static_cast<unsigned short>(byte)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A warp takes up to four pieces of 256 elements of a row, as above.
__global__ void __launch_bounds__(kQuantThreads)
    mxfp4_dequantize_kernel(const QuantArgs a, uint4* out) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int32_t L = rows_below(a.limit, a.rows);
  const int vecs = a.k / 8;
  const unsigned runs = (vecs + 32 * kQuantBatch - 1) / (32 * kQuantBatch);
  const int64_t units = static_cast<int64_t>(L) * runs;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kQuantWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kQuantWarps) {
    const int64_t r = units <= 0xFFFFFFFFll ? static_cast<unsigned>(u) / runs : u / runs;
    const int v0 = static_cast<int>(u - r * runs) * 32 * kQuantBatch + lane;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q + r * (a.k / 2));
    const uint8_t* s = a.scales + r * a.scale_width;
    uint32_t c[kQuantBatch], sb[kQuantBatch];
#pragma unroll
    for (int b = 0; b < kQuantBatch; ++b) {
      const int v = v0 + 32 * b;
      c[b] = v < vecs ? q[v] : 0u;
      sb[b] = v < vecs ? s[v >> 2] : 0u;
    }
#pragma unroll
    for (int b = 0; b < kQuantBatch; ++b) {
      if (v0 + 32 * b >= vecs) break;
      const float f = mx_scale(sb[b]);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = code_pair((c[b] >> (8 * i)) & 0xFFu);
        w[i] = pack_bf16x2(v.x * f, v.y * f);
      }
      out[r * vecs + v0 + 32 * b] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Weights [g, k, n] to rows along k: a thread owns one output column n and one block of 32 k.
// Reads are coalesced over n; each thread writes its 16 bytes of codes.
__global__ void __launch_bounds__(kQuantThreads)
    mxfp4_weights_kernel(const __nv_bfloat16* rhs, uint8_t* q,
                         uint8_t* scales, int32_t k, int32_t n, int32_t scale_width) {
  pdl_trigger();
  pdl_wait();
  const uint32_t col = blockIdx.x * kQuantThreads + threadIdx.x;  // up to a block past n: not in 31 bits
  const int block = blockIdx.y;
  const int64_t e = blockIdx.z;
  if (col >= static_cast<uint32_t>(n)) return;
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

// in 64 bits: the largest extents and a tile together leave 32
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// at most 24 blocks an SM (16381 rows of 4096, there and back: 8 an SM 57.9 us, 12 55.6, 24 53.9,
// 64 55.3: enough for an even end, few enough that the starts do not count)
int quant_grid(int64_t blocks, int sms) {
  const int64_t most = 24 * static_cast<int64_t>(sms);
  return static_cast<int>(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const QuantArgs& a, int sms, cudaStream_t stream) {
  const int64_t units = a.rows * ceil_div(a.k, 256 * kQuantBatch);
  const int grid = quant_grid(ceil_div(units, kQuantWarps), sms);
  return launch_pdl(a.pos != nullptr ? mxfp4_quantize_kernel<true> : mxfp4_quantize_kernel<false>,
                    dim3(grid), kQuantThreads, 0, 1, stream, a);
}

cudaError_t launch_mxfp4_dequantize(const QuantArgs& a, void* out, int sms, cudaStream_t stream) {
  const int64_t units = a.rows * ceil_div(a.k, 256 * kQuantBatch);
  return launch_pdl(mxfp4_dequantize_kernel, dim3(quant_grid(ceil_div(units, kQuantWarps), sms)),
                    kQuantThreads, 0, 1, stream, a, static_cast<uint4*>(out));
}

cudaError_t launch_mxfp4_quantize_weights(const void* rhs, uint8_t* q, uint8_t* scales, int32_t g,
                                          int32_t k, int32_t n, int32_t scale_width,
                                          cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(ceil_div(n, kQuantThreads)), scale_width, g);
  return launch_pdl(mxfp4_weights_kernel, grid, kQuantThreads, 0, 1, stream,
                    static_cast<const __nv_bfloat16*>(rhs), q, scales, k, n, scale_width);
}

}  // namespace rd
