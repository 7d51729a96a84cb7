// block_args.h -- host-side launchers of the norm, dropout, activation-gradient and linear kernels
// (the C entry points in api_block.cu check every argument first).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rd_block.h"
#include "wait_bound.h"

namespace rd {

struct NormArgs {
  const void* x;
  const void* d_out;     // backward
  const float* weight;   // [hidden] or null
  const float* bias;     // [hidden] or null
  void* out;             // forward: out; backward: d_x
  float* mean;           // [rows] or null (backward: input)
  float* rstd;
  float* d_weight;       // backward: [hidden] or null
  float* d_bias;
  float* parts;          // backward: workspace, [parts][2][hidden]
  const int32_t* limit;
  int32_t rows;
  int32_t hidden;
  int32_t split;         // backward: blocks that share a row too long for one (set by the launcher)
  int32_t split_cols;    // and the columns of each but the last
  float eps;
  WaitBound wait;        // backward: bound of the waits of blocks that share a row
};

cudaError_t launch_layer_norm_fwd(const NormArgs& a, int dtype, int out_dtype, int sms,
                                  cudaStream_t stream);
cudaError_t launch_layer_norm_bwd(const NormArgs& a, int dtype, int out_dtype, int sms,
                                  cudaStream_t stream);
// rows of partial sums that the backward pass keeps in its workspace
int layer_norm_bwd_parts(int64_t rows, int64_t hidden, int sms);
// whether it is the kernel for few rows, which needs no workspace
bool layer_norm_bwd_few(int64_t rows, int64_t hidden);

struct DropoutArgs {
  const void* x;
  const void* residual;  // or null
  void* out;
  const int64_t* rng;
  const int32_t* limit;
  int32_t rows;
  int32_t vecs;          // 8-element vectors of a row
  int32_t least;         // smallest 16 bits that keep an element
  float scale;
};

cudaError_t launch_dropout_rows(const DropoutArgs& a, int dtype, int out_dtype, int sms,
                                cudaStream_t stream);

struct ActBwdArgs {
  const void* d_out;
  const void* pre;       // bf16 or null (no activation)
  void* d_pre;           // bf16 or null
  float* d_bias;         // [g_local, n] or null
  float* parts;          // workspace: boundaries, then the sums [shares + groups][n]
  const int32_t* group_sizes;  // or null: one group of all rows
  const int32_t* limit;
  int32_t* status;
  int32_t m;
  int32_t n;
  int32_t g_total;
  int32_t group_offset;
  int32_t g_local;
  int32_t act;
  int32_t shares;        // of the rows, a block's each (set by the launcher)
};

cudaError_t launch_linear_act_bwd(const ActBwdArgs& a, int out_dtype, int sms, cudaStream_t stream);
// bytes of its workspace
int64_t linear_act_bwd_bytes(int64_t m, int64_t n, int32_t g_local);

}  // namespace rd
