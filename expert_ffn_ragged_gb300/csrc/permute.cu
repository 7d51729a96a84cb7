// permute.cu -- token rows to packed rows (dispatch), back (combine), and combine's gradients.
//
// All three are streams of 16-byte vectors.  A warp owns a piece of a token's row (dispatch,
// combine) or a whole row of a slot (the gradients, whose dot product it then reduces alone).
// Packed rows are found through pos, so no inverse permutation is needed and x, d_out and out
// cross HBM once.
//
// Bound: HBM.  dispatch, 28160 tokens top-8 of 4096: 2.08 GB in 306 us (6.79 TB/s, the plain copy's rate);
// combine, 16384 tokens top-2: 403 MB in 62.4 us (6.5 TB/s); the gradients, 15769 tokens top-8: 2.20 GB
// in 321 us (6.84 TB/s).  16 tokens top-8 combine in 2.8 us, a launch and one trip to memory.
#include <cuda_runtime.h>
#include <stdint.h>

#include "glu_math.cuh"
#include "launch.h"
#include "moe_args.h"

namespace rd {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowBatch = 4;  // vectors per lane of one piece

__device__ __forceinline__ int32_t rows_below(const int32_t* limit, int32_t rows) {
  if (limit == nullptr) return rows;
  const int32_t v = *limit;
  return v < 0 ? 0 : (v > rows ? rows : v);
}

__device__ __forceinline__ uint4 ld_row(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__global__ void __launch_bounds__(kRowThreads) dispatch_rows_kernel(const RowsArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int32_t L = rows_below(a.limit, a.tokens);
  const int pieces = (a.vecs + 32 * kRowBatch - 1) / (32 * kRowBatch);
  const int64_t units = static_cast<int64_t>(L) * pieces;
  const uint4* x = static_cast<const uint4*>(a.x);
  uint4* out = static_cast<uint4*>(a.out);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    const int64_t t = u / pieces;
    const int v0 = static_cast<int>(u - t * pieces) * 32 * kRowBatch + lane;
    const int32_t p_lane = lane < a.topk ? a.pos[t * a.topk + lane] : -1;
    uint4 v[kRowBatch];
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b)
      if (v0 + 32 * b < a.vecs) v[b] = ld_row(x + t * a.vecs + v0 + 32 * b);
    for (int k = 0; k < a.topk; ++k) {
      const int32_t p = __shfl_sync(0xFFFFFFFFu, p_lane, k);
      if (p < 0 || p >= a.packed_rows) continue;
      uint4* o = out + static_cast<int64_t>(p) * a.vecs;
#pragma unroll
      for (int b = 0; b < kRowBatch; ++b)
        if (v0 + 32 * b < a.vecs) o[v0 + 32 * b] = v[b];
    }
  }
}

__device__ __forceinline__ void add_scaled(float (&acc)[8], uint4 y, float w) {
  const uint32_t c[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(w, bf16_lo(c[i]), acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, bf16_hi(c[i]), acc[2 * i + 1]);
  }
}

// A warp owns B * 32 vectors of a token's row; the rows of S slots are in flight at once.
template <int B, int S>
__global__ void __launch_bounds__(kRowThreads) combine_rows_kernel(const RowsArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int32_t L = rows_below(a.limit, a.tokens);
  const int pieces = (a.vecs + 32 * B - 1) / (32 * B);
  const int64_t units = static_cast<int64_t>(L) * pieces;
  const uint4* y = static_cast<const uint4*>(a.x);
  uint4* out = static_cast<uint4*>(a.out);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    const int64_t t = u / pieces;
    const int v0 = static_cast<int>(u - t * pieces) * 32 * B + lane;
    int32_t p_lane = -1;
    float w_lane = 0.0f;
    if (lane < a.topk) {
      p_lane = a.pos[t * a.topk + lane];
      w_lane = a.w != nullptr ? a.w[t * a.topk + lane] : 1.0f;
    }
    float acc[B][8];
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[b][i] = 0.0f;
    for (int k0 = 0; k0 < a.topk; k0 += S) {
      uint4 v[S][B];
      float w[S];
      bool on[S];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int32_t p = __shfl_sync(0xFFFFFFFFu, p_lane, (k0 + i) & 31);
        w[i] = __shfl_sync(0xFFFFFFFFu, w_lane, (k0 + i) & 31);
        on[i] = k0 + i < a.topk && p >= 0 && p < a.packed_rows;
        if (on[i]) {
#pragma unroll
          for (int b = 0; b < B; ++b)
            if (v0 + 32 * b < a.vecs) v[i][b] = ld_row(y + static_cast<int64_t>(p) * a.vecs + v0 + 32 * b);
        }
      }
#pragma unroll
      for (int i = 0; i < S; ++i) {
        if (on[i]) {
#pragma unroll
          for (int b = 0; b < B; ++b)
            if (v0 + 32 * b < a.vecs) add_scaled(acc[b], v[i][b], w[i]);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (v0 + 32 * b < a.vecs)
        out[t * a.vecs + v0 + 32 * b] =
            make_uint4(pack_bf16x2(acc[b][0], acc[b][1]), pack_bf16x2(acc[b][2], acc[b][3]),
                       pack_bf16x2(acc[b][4], acc[b][5]), pack_bf16x2(acc[b][6], acc[b][7]));
  }
}

__device__ __forceinline__ uint32_t scale_dot(uint32_t d, uint32_t y, float w, float& dot) {
  const float d0 = bf16_lo(d), d1 = bf16_hi(d);
  dot = fmaf(d0, bf16_lo(y), dot);
  dot = fmaf(d1, bf16_hi(y), dot);
  return pack_bf16x2(__fmul_rn(d0, w), __fmul_rn(d1, w));
}

__global__ void __launch_bounds__(kRowThreads) combine_rows_bwd_kernel(const RowsArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int32_t L = rows_below(a.limit, a.tokens);
  const int64_t slots = static_cast<int64_t>(L) * a.topk;
  const uint4* d_out = static_cast<const uint4*>(a.x);
  const uint4* y = static_cast<const uint4*>(a.y);
  uint4* d_y = static_cast<uint4*>(a.out);
  for (int64_t s = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); s < slots;
       s += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    const int64_t t = s / a.topk;
    const int32_t p = a.pos[s];
    float dot = 0.0f;
    if (p >= 0 && p < a.packed_rows) {
      const float w = a.w[s];
      const uint4* dr = d_out + t * a.vecs;
      const uint4* yr = y + static_cast<int64_t>(p) * a.vecs;
      uint4* o = d_y + static_cast<int64_t>(p) * a.vecs;
      for (int v0 = lane; v0 < a.vecs; v0 += 32 * kRowBatch) {
        uint4 dv[kRowBatch], yv[kRowBatch];
#pragma unroll
        for (int b = 0; b < kRowBatch; ++b) {
          if (v0 + 32 * b < a.vecs) {
            dv[b] = dr[v0 + 32 * b];
            yv[b] = ld_row(yr + v0 + 32 * b);
          }
        }
#pragma unroll
        for (int b = 0; b < kRowBatch; ++b)
          if (v0 + 32 * b < a.vecs)
            o[v0 + 32 * b] = make_uint4(scale_dot(dv[b].x, yv[b].x, w, dot), scale_dot(dv[b].y, yv[b].y, w, dot),
                                        scale_dot(dv[b].z, yv[b].z, w, dot), scale_dot(dv[b].w, yv[b].w, w, dot));
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
    }
    if (lane == 0) a.d_w[s] = dot;
  }
}

// Blocks of a launch: at most `per_sm` for each SM, which the warps then stride through.  Many short
// blocks are handed out in order and keep the rows in flight close together, which the scattered
// writes of dispatch and of combine's gradient gain from (28160 tokens top-8 of 4096: 8 blocks an SM
// 328 us, 24 319, 64 309, 128 306; the gradient at 15769 tokens: 337, 328, 322, 322); combine only
// pays for the starts (16384 tokens top-2: 62, 64, 67, 71 us).
constexpr int kDispatchBlocks = 128;
constexpr int kCombineBlocks = 8;
constexpr int kCombineBwdBlocks = 64;

int row_grid(int64_t units, int sms, int per_sm) {
  const int64_t blocks = (units + kRowWarps - 1) / kRowWarps;
  const int64_t most = static_cast<int64_t>(per_sm) * sms;
  return static_cast<int>(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_dispatch_rows(const RowsArgs& a, int sms, cudaStream_t stream) {
  const int64_t pieces = (a.vecs + 32 * kRowBatch - 1) / (32 * kRowBatch);
  return launch_pdl(dispatch_rows_kernel, dim3(row_grid(a.tokens * pieces, sms, kDispatchBlocks)), kRowThreads, 0, 1, stream, a);
}

cudaError_t launch_combine_rows(const RowsArgs& a, int sms, cudaStream_t stream) {
  // Enough work for every warp of the GPU (64 an SM): two vectors a lane and two slots at once.
  // Less: one vector, so that a few tokens spread over more SMs, and up to four slots, since a warp
  // has little else to hide a load behind.
  const int64_t twos = static_cast<int64_t>(a.tokens) * ((a.vecs + 63) / 64);
  if (twos >= 64 * static_cast<int64_t>(sms))
    return launch_pdl(combine_rows_kernel<2, 2>, dim3(row_grid(twos, sms, kCombineBlocks)), kRowThreads, 0, 1, stream, a);
  const int64_t ones = static_cast<int64_t>(a.tokens) * ((a.vecs + 31) / 32);
  return launch_pdl(a.topk > 2 ? combine_rows_kernel<1, 4> : combine_rows_kernel<1, 2>,
                    dim3(row_grid(ones, sms, kCombineBlocks)), kRowThreads, 0, 1, stream, a);
}

cudaError_t launch_combine_rows_bwd(const RowsArgs& a, int sms, cudaStream_t stream) {
  return launch_pdl(combine_rows_bwd_kernel, dim3(row_grid(static_cast<int64_t>(a.tokens) * a.topk, sms, kCombineBwdBlocks)),
                    kRowThreads, 0, 1, stream, a);
}

}  // namespace rd
