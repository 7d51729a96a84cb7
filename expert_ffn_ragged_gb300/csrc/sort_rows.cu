// sort_rows.cu -- the plan of the packed buffer: a stable counting sort of the slots by expert.
//
// pos of a slot = (slots of lower experts) + (earlier slots of the same expert).  One cluster of
// up to 16 CTAs does the whole sort in one launch: every warp counts a contiguous piece of the
// slots into its own histogram in shared memory, the CTAs exchange their sums through distributed
// shared memory, and every warp then walks its piece again, 32 slots at a time: each slot sets its
// lane's bit in a mask of its expert, whose lower bits then count the slots before it.  The ids are
// read twice (the second time from L2) and pos is written once: 4 + 4 bytes a slot.
//
// Bound: latency, that of the walk's dependent steps.  Each warp therefore loads eight steps' ids
// before it works on them (a load a step made 262144 slots take 40 us on 8 CTAs), and the cluster
// grows with the slots until a warp has one such batch.  The walk of 262168 slots over 256 experts
// took 17 us with a warp match for equal experts (60 cycles a step of a whole SM) and 12 us with
// a ballot per bit of the index.  262168 slots over 256 experts: 15.1 us in all, 8 slots: 4.4 us.  Two
// launches over all SMs, the counts passed through memory, saved 2 us there and cost 0.2 us where a call
// is small.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "launch.h"
#include "moe_args.h"

namespace cg = cooperative_groups;

namespace rd {
namespace {

constexpr int kSortWarps = 32;    // warps of a CTA up to kSortWide experts, half as many above
constexpr int kSortWide = 512;    // (the warps' counts and masks have to fit in shared memory)
constexpr int kSortBatch = 8;     // steps (of 32 slots) whose ids a warp loads at once
constexpr int kSortCluster = 16;  // most CTAs of a sort (one cluster; above 8 by opt-in)

template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32)
    sort_rows_kernel(const int32_t* ids, int32_t tokens, int32_t topk, int32_t experts,
                     const int32_t* limit, int32_t* group_sizes,
                     int32_t* pos, int32_t* rows) {
  // [warps][experts] counts, then first positions; [warps][experts] lane masks; [experts] the
  // CTA's sums; [experts] first rows
  extern __shared__ uint32_t smem[];
  uint32_t* hist = smem;
  uint32_t* masks = hist + WARPS * experts;
  uint32_t* sums = masks + WARPS * experts;
  uint32_t* base = sums + experts;
  __shared__ uint32_t warp_total[32];
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  int32_t L = tokens;
  if (limit != nullptr) {
    const int32_t v = *limit;
    L = v < 0 ? 0 : (v > tokens ? tokens : v);
  }
  const int64_t slots = static_cast<int64_t>(L) * topk;
  // pieces of whole 32-slot steps
  const int64_t steps = (slots + 31) / 32;
  const int64_t per = (steps + ctas * WARPS - 1) / (ctas * WARPS);
  const int64_t piece = static_cast<int64_t>(rank) * WARPS + warp;
  const int64_t s0 = min(piece * per, steps), s1 = min(s0 + per, steps);
  uint32_t* mine = hist + warp * experts;
  uint32_t* mask = masks + warp * experts;

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
  for (int i = lane; i < experts; i += 32) mine[i] = mask[i] = 0;
  __syncwarp();
  for (int64_t s = s0; s < s1; s += kSortBatch) {
    if (s != s0) load(s, e);
#pragma unroll
    for (int b = 0; b < kSortBatch; ++b)
      if (e[b] >= 0) atomicAdd(&mine[e[b]], 1u);  // counts only: the order does not matter
  }
  __syncthreads();
  // exclusive prefix over the CTA's warps, and the CTA's sum, of each expert
  for (int x = tid; x < experts; x += WARPS * 32) {
    uint32_t run = 0;
#pragma unroll 8
    for (int w = 0; w < WARPS; ++w) {
      const uint32_t c = hist[w * experts + x];
      hist[w * experts + x] = run;
      run += c;
    }
    sums[x] = run;
  }
  cluster.sync();
  // sums of all CTAs, and of those before this one: two neighbouring experts a thread
  uint32_t total[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int x = 2 * tid + i;
    if (x >= experts) continue;
#pragma unroll 4
    for (unsigned c = 0; c < ctas; ++c) {
      const uint32_t v = cluster.map_shared_rank(sums, c)[x];
      if (c < rank) before[i] += v;
      total[i] += v;
    }
  }
  // exclusive prefix of the totals over the experts
  const uint32_t both = total[0] + total[1];
  uint32_t incl = both;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  uint32_t first_row = incl - both, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const uint32_t v = warp_total[w];
    if (w < warp) first_row += v;
    all += v;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int x = 2 * tid + i;
    if (x >= experts) continue;
    base[x] = first_row + (i > 0 ? total[0] : 0u) + before[i];
    if (rank == 0) group_sizes[x] = static_cast<int32_t>(total[i]);
  }
  if (rank == 0 && tid == 0) rows[0] = static_cast<int32_t>(all);
  __syncthreads();
  const bool one_batch = s1 - s0 <= kSortBatch;  // its ids are still here
  for (int64_t s = s0; s < s1; s += kSortBatch) {
    if (!one_batch) load(s, e);
#pragma unroll
    for (int b = 0; b < kSortBatch; ++b) {
      if (s + b >= s1) break;
      const bool live = e[b] >= 0;
      if (live) atomicOr(&mask[e[b]], 1u << lane);
      __syncwarp();
      uint32_t peers = 0, first = 0;
      if (live) {
        peers = mask[e[b]];
        first = mine[e[b]];
      }
      const int before_me = __popc(peers & ((1u << lane) - 1u));
      __syncwarp();
      if (live && before_me == 0) {
        mine[e[b]] = first + __popc(peers);
        mask[e[b]] = 0;
      }
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
  const bool wide = experts > kSortWide;
  const int warps = wide ? kSortWarps / 2 : kSortWarps;
  const auto kernel = wide ? sort_rows_kernel<kSortWarps / 2> : sort_rows_kernel<kSortWarps>;
  static std::atomic<bool> attr_set[2][64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[wide][dev].load(std::memory_order_acquire)) {
    const size_t most = sizeof(uint32_t) * (2 * warps + 2) * (wide ? RD_MAX_GROUPS : kSortWide);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(most));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set[wide][dev].store(true, std::memory_order_release);
  }
  // the smallest power of two of CTAs that gives every warp one batch, at most 16
  const int64_t slots = static_cast<int64_t>(tokens) * topk;
  int ctas = 1;
  while (ctas < kSortCluster && slots > static_cast<int64_t>(ctas) * warps * 32 * kSortBatch) ctas *= 2;
  return launch_pdl(kernel, dim3(ctas), warps * 32, sizeof(uint32_t) * (2 * warps + 2) * experts, ctas,
                    stream, ids, tokens, topk, experts, limit, group_sizes, pos, rows);
}

}  // namespace rd
