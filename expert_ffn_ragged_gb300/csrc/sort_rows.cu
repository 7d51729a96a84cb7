// sort_rows.cu -- the plan of the packed buffer: a stable counting sort of the slots by expert.
//
// pos of a slot = (slots of lower experts) + (earlier slots of the same expert).  One cluster of
// up to 16 CTAs does the whole sort in one launch: every warp counts a contiguous piece of the
// slots into its own histogram in shared memory, the CTAs exchange their sums through distributed
// shared memory, and every warp then walks its piece again, 32 slots at a time, ranking equal
// experts among the lanes with a warp match.  The ids are read twice (the second time from L2)
// and pos is written once: 4 + 4 bytes a slot.
//
// Bound: latency, that of the walk's dependent steps.  Each warp therefore loads eight steps' ids
// before it works on them (a load a step made 262144 slots take 40 us on 8 CTAs), and the cluster
// grows with the slots until a warp has one such batch.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "moe_args.h"

namespace cg = cooperative_groups;

namespace rd {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBatch = 8;     // steps (of 32 slots) whose ids a warp loads at once
constexpr int kSortCluster = 16;  // most CTAs of a sort (one cluster; above 8 by opt-in)

__global__ void __launch_bounds__(kSortThreads)
    sort_rows_kernel(const int32_t* __restrict__ ids, int32_t tokens, int32_t topk, int32_t experts,
                     const int32_t* limit, int32_t* __restrict__ group_sizes,
                     int32_t* __restrict__ pos, int32_t* __restrict__ rows) {
  // [warps][experts] counts, then first positions; [experts] the CTA's sums; [experts] first rows
  extern __shared__ uint32_t smem[];
  uint32_t* hist = smem;
  uint32_t* sums = smem + kSortWarps * experts;
  uint32_t* base = sums + experts;
  __shared__ uint32_t warp_total[32];
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t L = tokens;
  if (limit != nullptr) {
    const int32_t v = *limit;
    L = v < 0 ? 0 : (v > tokens ? tokens : v);
  }
  const int64_t slots = static_cast<int64_t>(L) * topk;
  // pieces of whole 32-slot steps
  const int64_t steps = (slots + 31) / 32;
  const int64_t per = (steps + ctas * kSortWarps - 1) / (ctas * kSortWarps);
  const int64_t piece = static_cast<int64_t>(rank) * kSortWarps + warp;
  const int64_t s0 = min(piece * per, steps), s1 = min(s0 + per, steps);
  uint32_t* mine = hist + warp * experts;

  // the ids of up to eight steps from s on; -1 for a slot without an expert
  auto load = [&](int64_t s, int32_t (&e)[kSortBatch]) {
#pragma unroll
    for (int b = 0; b < kSortBatch; ++b) {
      const int64_t i = (s + b) * 32 + lane;
      int32_t v = -1;
      if (s + b < s1 && i < slots) v = ids[i];
      e[b] = v < experts ? v : -1;
    }
  };

  int32_t e[kSortBatch];
  load(s0, e);
  for (int i = lane; i < experts; i += 32) mine[i] = 0;
  __syncwarp();
  for (int64_t s = s0; s < s1; s += kSortBatch) {
    if (s != s0) load(s, e);
#pragma unroll
    for (int b = 0; b < kSortBatch; ++b)
      if (e[b] >= 0) atomicAdd(&mine[e[b]], 1u);  // counts only: the order does not matter
  }
  __syncthreads();
  // exclusive prefix over the CTA's warps, and the CTA's sum, of each expert
  for (int x = tid; x < experts; x += kSortThreads) {
    uint32_t run = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = hist[w * experts + x];
      hist[w * experts + x] = run;
      run += c;
    }
    sums[x] = run;
  }
  cluster.sync();
  // sums of all CTAs, and of those before this one (experts <= the thread count: one each)
  uint32_t total = 0, before = 0;
  if (tid < experts) {
#pragma unroll 4
    for (unsigned c = 0; c < ctas; ++c) {
      const uint32_t v = cluster.map_shared_rank(sums, c)[tid];
      if (c < rank) before += v;
      total += v;
    }
  }
  // exclusive prefix of the totals over the experts
  uint32_t incl = total;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    uint32_t v = warp_total[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v += o;
    }
    warp_total[lane] = v;
  }
  __syncthreads();
  if (tid < experts) {
    base[tid] = incl - total + (warp > 0 ? warp_total[warp - 1] : 0u) + before;
    if (rank == 0) group_sizes[tid] = static_cast<int32_t>(total);
  }
  if (rank == 0 && tid == 0) rows[0] = static_cast<int32_t>(warp_total[31]);
  __syncthreads();
  const bool one_batch = s1 - s0 <= kSortBatch;  // its ids are still here
  for (int64_t s = s0; s < s1; s += kSortBatch) {
    if (!one_batch) load(s, e);
#pragma unroll
    for (int b = 0; b < kSortBatch; ++b) {
      if (s + b >= s1) break;
      const unsigned peers = __match_any_sync(0xFFFFFFFFu, e[b]);
      const int before_me = __popc(peers & ((1u << lane) - 1u));
      uint32_t first = 0;
      if (e[b] >= 0) first = mine[e[b]];
      __syncwarp();
      if (e[b] >= 0 && before_me == 0) mine[e[b]] = first + __popc(peers);
      __syncwarp();
      const int64_t i = (s + b) * 32 + lane;
      if (i < slots) pos[i] = e[b] >= 0 ? static_cast<int32_t>(base[e[b]] + first + before_me) : -1;
    }
  }
  cluster.sync();  // no CTA leaves while another still reads its sums
}

}  // namespace

cudaError_t launch_sort_rows(const int32_t* ids, int32_t tokens, int32_t topk, int32_t experts,
                             const int32_t* limit, int32_t* group_sizes, int32_t* pos,
                             int32_t* rows, cudaStream_t stream) {
  const size_t most = sizeof(uint32_t) * (kSortWarps + 2) * RD_MAX_GROUPS;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(sort_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(most));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(sort_rows_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  // the smallest power of two of CTAs that gives every warp one batch, at most 16
  const int64_t slots = static_cast<int64_t>(tokens) * topk;
  int ctas = 1;
  while (ctas < kSortCluster && slots > static_cast<int64_t>(ctas) * kSortThreads * kSortBatch) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kSortThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(uint32_t) * (kSortWarps + 2) * experts;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sort_rows_kernel, ids, tokens, topk, experts, limit, group_sizes,
                            pos, rows);
}

}  // namespace rd
