// gemm_split.h -- launch arguments of the product for few output tiles (gemm_split.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "wait_bound.h"

namespace rd {

struct SplitArgs {
  const float* bias;      // [n] or null
  const void* residual;   // [m, n] of the output's type or null
  void* out;              // [m, n] bf16 or f32
  void* pre;              // [m, n] bf16 or null
  const int32_t* group_sizes;  // or null: one weight
  const int32_t* limit;
  int32_t* status;
  int32_t m;
  int32_t k;
  int32_t n;
  int32_t act;
  int32_t g_total;        // (with group_sizes)
  int32_t group_offset;
  int32_t g_local;
  int32_t row_tiles;      // of the grid: the most that the rows can fill
  int32_t box_rows;       // rows of an output tile and of x's boxes (multiple of 8, at most kSplitRows)
  int32_t stages;
  int32_t ring_bytes;     // of shared memory for the stages: kSplitRing or kSplitRingAlone
  int32_t cluster;        // CTAs that share one output tile's k
  WaitBound wait;         // bound of every wait inside the kernel
};

constexpr int kSplitMaxStages = 12;
constexpr int kSplitRows = 128;    // rows of an MMA, and most rows of an output tile
// rings that leave room for two CTAs on an SM, and for one
constexpr int kSplitRing = 108 * 1024;
constexpr int kSplitRingAlone = 216 * 1024;

// columns of an output tile: 64 or 128
cudaError_t launch_gemm_split(bool f32_out, int cols, const CUtensorMap& tmap_x, const CUtensorMap& tmap_w,
                              const SplitArgs& args, cudaStream_t stream);

}  // namespace rd
