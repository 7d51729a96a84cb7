// moe_args.h -- host-side launchers of the routing, sorting, dispatch, combine and 4-bit row
// kernels (the C entry points in api_moe.cu check every argument first).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rd_moe.h"

namespace rd {

struct RouteArgs {
  const void* logits;    // [tokens, experts]
  const float* bias;     // [experts] or null
  const int32_t* limit;  // device scalar or null
  int32_t* ids;          // [tokens, topk] (backward: input)
  float* weights;        // [tokens, topk]
  const float* d_weights;
  void* d_logits;
  int32_t tokens;
  int32_t experts;
  int32_t topk;
  int32_t groups;
  int32_t topk_groups;
  int32_t score;
  int32_t renormalize;
  float scale;
  bool vec;              // rows start on vector boundaries (set by the launcher)
};

cudaError_t launch_route(const RouteArgs& a, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_route_bwd(const RouteArgs& a, int dtype, int sms, cudaStream_t stream);

cudaError_t launch_sort_rows(const int32_t* ids, int32_t tokens, int32_t topk, int32_t experts,
                             const int32_t* limit, int32_t* group_sizes, int32_t* pos,
                             int32_t* rows, cudaStream_t stream);

// rows [0, L) of one matrix and the packed rows that their slots stand for
struct RowsArgs {
  const void* x;         // dispatch: x; combine: y; backward: d_out
  const void* y;         // backward: y
  const int32_t* pos;    // [tokens, topk]
  const float* w;        // [tokens, topk] or null
  void* out;             // dispatch / combine: out; backward: d_y
  float* d_w;
  const int32_t* limit;
  int32_t tokens;
  int32_t topk;
  int32_t vecs;          // 16-byte vectors of a row
  int32_t packed_rows;   // rows of the packed matrix (positions outside are skipped)
};

cudaError_t launch_dispatch_rows(const RowsArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_combine_rows(const RowsArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_combine_rows_bwd(const RowsArgs& a, int sms, cudaStream_t stream);

struct QuantArgs {
  const void* x;         // [rows, k] bf16 (dequantize: out)
  const int32_t* pos;    // [rows, topk] or null
  uint8_t* q;
  uint8_t* scales;
  const int32_t* limit;
  int32_t rows;
  int32_t topk;
  int32_t k;
  int32_t scale_width;
  int32_t out_rows;
};

cudaError_t launch_mxfp4_quantize(const QuantArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_mxfp4_dequantize(const QuantArgs& a, void* out, int sms, cudaStream_t stream);
cudaError_t launch_mxfp4_quantize_weights(const void* rhs, uint8_t* q, uint8_t* scales, int32_t g,
                                          int32_t k, int32_t n, int32_t scale_width,
                                          cudaStream_t stream);

struct Gemm4Maps;
struct Gemm4Args;
cudaError_t launch_gemm_mxfp4(int epi, int variant, const Gemm4Maps& maps, const Gemm4Args& args,
                              int grid, cudaStream_t stream);

}  // namespace rd
