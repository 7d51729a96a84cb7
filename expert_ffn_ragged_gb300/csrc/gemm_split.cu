// gemm_split.cu -- rd_linear with few output tiles: a decoding batch, of one weight or by expert, whose time is the
// weights' bytes, or a router's few columns, whose time is the tokens'.
//
// The persistent kernel (gemm_kernel.cuh) gives an output tile to one CTA (pair), so with few tiles most SMs
// would stand still.  Here an output tile of 128 rows x 64 or 128 columns belongs to a cluster of up to
// eight CTAs that share its k: each streams its part of the weights through its own ring (TMA, 128-byte
// swizzle) into a tcgen05 accumulator, writes the f32 sums to shared memory, and after a cluster barrier
// each adds its share of the tile over the cluster's CTAs, in their order, through distributed shared memory; bias,
// activation and residual follow in f32.  No workspace, no atomics, no second launch.  Two CTAs fit an SM, so
// that one's set-up and epilogue overlap the other's copies, and all CTAs of a call usually run at once: the
// copies of all of them together are what HBM sees.
//
// An f32 output (a router's logits) is kept as exact as a sum in f32 with rounding: the tensor core cuts its sums off
// after every step of 16 along k (16381 x 4096 x 128: 4.3e-6 of the result's norm off, 6e-7 for rounded sums), so every 512
// of k the accumulator changes and four warps add the complete one to sums in registers, while the MMAs go on.
//
// Bound: HBM.  1 x 4096 x 14336, bf16: 118 MB in 21.9 us (5.4 TB/s; with k = 32768 6.6), 64 x 14336 x 4096 with a residual 120 MB in
// 23.5, 16381 x 4096 x 128, f32: 144 MB in 29.8 (4.8 TB/s).  Without any MMA they take 20.9, 22.6 and 28.1: what is left is the start of
// the copies, the last tile and, for the last of the three, 128 tiles for 152 SMs; the weights, which every SM reads from L2 there,
// cost nothing.
//
// By group the grid has as many row tiles as the rows can fill; each CTA adds the group sizes up, finds its tile, or none and leaves,
// and sets its share of the rows outside the local groups to zero.
//
// The MMA always has 128 rows; x brings only box_rows of them, and the rest of the operand's rows are whatever
// lies behind in shared memory: their products land in accumulator rows that nothing reads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "act_math.cuh"
#include "gemm_split.h"
#include "launch.h"
#include "ptx.cuh"
#include "rows.cuh"
#include "schedule.h"

namespace rd {
namespace {

constexpr int kSplitThreads = 256;  // warp 0 copies, warp 1 issues the MMAs; all eight take the sums
constexpr WaitBound kSplitDrain = wait_bound(1000000000ull);
constexpr int kStretch = 8;  // K blocks that the tensor core sums before an f32 output takes them over

struct SplitShared {
  uint64_t full[kSplitMaxStages];
  uint64_t empty[kSplitMaxStages];
  uint64_t done;
  uint64_t tfull[2];   // f32 outputs: the accumulator of a stretch of k is complete, or has been read
  uint64_t tempty[2];
  uint32_t tmem_base;
  int32_t abort_flag;
  // by group: this CTA's tile (group, first row, end of the group's rows) and the rows outside the local groups
  int32_t group, row0, group_end, zero_lo, zero_hi;
};

constexpr size_t split_smem(int ring_bytes) { return 1024 + ring_bytes + sizeof(SplitShared); }

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <class O>
struct IsF32 {
  static constexpr bool value = false;
};
template <>
struct IsF32<float> {
  static constexpr bool value = true;
};

// Run by one warp: row tile t of the local groups' tiles in order, box_rows high.
__device__ __forceinline__ void find_tile(SplitShared& sh, const SplitArgs& a, int32_t L, int t, int lane) {
  const int G = a.g_total, per = (G + 31) / 32, lo = min(lane * per, G), hi = min(lo + per, G);
  long long sum = 0;
  bool neg = false;
  for (int i = lo; i < hi; ++i) {
    const int32_t s = a.group_sizes[i];
    neg |= s < 0;
    sum += s > 0 ? s : 0;
  }
  long long incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += o;
  }
  const long long total = __shfl_sync(0xFFFFFFFFu, incl, 31);
  neg = __any_sync(0xFFFFFFFFu, neg);
  if (lane == 0) sh.group = sh.row0 = sh.group_end = 0;
  __syncwarp();
  // once to count this lane's tiles, once to find the one that is wanted
  int before = 0, tiles = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    long long run = incl - sum;
    int at = before;
    for (int i = lo; i < hi; ++i) {
      const int32_t s = a.group_sizes[i], b0 = clamp_boundary(run, L);
      run += s > 0 ? s : 0;
      const int32_t b1 = clamp_boundary(run, L), j = i - a.group_offset;
      if (j < 0 || j >= a.g_local) continue;
      const int n = ceil_div(b1 - b0, a.box_rows);
      if (pass == 0) {
        if (j == 0) sh.zero_lo = b0;
        if (j == a.g_local - 1) sh.zero_hi = b1;
      } else if (t >= at && t < at + n) {
        sh.group = j;
        sh.row0 = b0 + (t - at) * a.box_rows;
        sh.group_end = b1;
      }
      at += n;
    }
    if (pass == 0) {
      tiles = at;
      int upto = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += o;
      }
      before = upto - tiles;
    }
  }
  if (lane == 0 && a.status != nullptr && blockIdx.x == 0 && blockIdx.y == 0) {
    const int bits = (neg ? RD_STATUS_NEG_SIZE : 0) | (total > a.m ? RD_STATUS_OVERFLOW : 0);
    if (bits) atomicOr(a.status, bits);
  }
}

// +0 in the rows outside the local groups: 64 threads of every CTA
__device__ __forceinline__ void zero_rows(const SplitShared& sh, int32_t L, void* out, int64_t row_bytes, int thread) {
  const int64_t vecs = row_bytes / 16, low = sh.zero_lo * vecs, all = low + (L - sh.zero_hi) * vecs;
  const int64_t step = static_cast<int64_t>(gridDim.x) * gridDim.y * 64;
  uint4* p = static_cast<uint4*>(out);
  for (int64_t v = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 64 + thread; v < all; v += step)
    p[v < low ? v : v - low + sh.zero_hi * vecs] = make_uint4(0, 0, 0, 0);
}

// C: CTAs that share a tile's k; G: by group (else one weight for all rows)
template <class O, int BN, int C, bool G>
__global__ void __launch_bounds__(kSplitThreads, IsF32<O>::value && BN == 128 ? 1 : 2)
    gemm_split_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                      const SplitArgs a) {
  constexpr bool kFine = IsF32<O>::value;
  constexpr uint32_t kTmem = kFine ? 2 * BN : BN;  // columns
  constexpr int kPitch = BN + 4;  // floats between rows of the staged sums: no bank conflicts
  static_assert(kSplitRows * kPitch * 4 <= kSplitRing, "the staged sums take the ring's place");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  SplitShared& sh = *reinterpret_cast<SplitShared*>(smem + a.ring_bytes);
  const uint32_t a_bytes = static_cast<uint32_t>(a.box_rows) * 128;
  constexpr uint32_t b_bytes = BN * kBK * 2;
  uint8_t* s_a = smem;
  uint8_t* s_b = smem + a.stages * a_bytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sh.abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      ptx::mbar_init(ptx::smem_addr(&sh.full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh.empty[s]), 1);
    }
    ptx::mbar_init(ptx::smem_addr(&sh.done), 1);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_addr(&sh.tfull[b]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh.tempty[b]), 4);
    }
    sh.abort_flag = 0;
    ptx::fence_mbar_init();
    if (a.k > 0) {  // (else there are no maps)
      ptx::prefetch_tmap(&tmap_x);
      ptx::prefetch_tmap(&tmap_w);
    }
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(&sh.tmem_base), kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  pdl_trigger();
  pdl_wait();

  const int rank = static_cast<int>(blockIdx.x) % C;
  const int32_t col0 = static_cast<int32_t>(blockIdx.x) / C * BN;
  const int32_t L = rows_within(a.limit, a.m);
  int32_t row0 = static_cast<int32_t>(blockIdx.y) * a.box_rows, group_end = L, group = 0;
  if constexpr (G) {
    if (warp == 2) find_tile(sh, a, L, static_cast<int>(blockIdx.y), lane);
    __syncthreads();
    row0 = sh.row0;
    group_end = sh.group_end;
    group = sh.group;
  }
  const float* const bias_row = a.bias == nullptr ? nullptr : a.bias + static_cast<int64_t>(group) * a.n;
  const int32_t row_end = group_end - row0 > a.box_rows ? row0 + a.box_rows : group_end;  // rows [row0, row_end) are stored
  const bool live = row_end > row0;                                       // the same in the whole cluster
  // the box ends at row_end, so that no row at or past L is read (rows before 0 arrive as zeros, rows of the group in front are
  // not stored)
  const int32_t row_load = row_end - a.box_rows;
  const int nkb = ceil_div(a.k, kBK);
  const int kb0 = static_cast<int>(static_cast<int64_t>(nkb) * rank / C);
  const int kb1 = live ? static_cast<int>(static_cast<int64_t>(nkb) * (rank + 1) / C) : kb0;
  int fills = 0;               // stages that this thread has filled: the first thread's
  float sums[kFine ? BN : 1];  // of a row, in warps 4 to 7

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        const uint32_t bar = ptx::smem_addr(&sh.full[stage]);
        if (!ptx::mbar_wait_bounded(ptx::smem_addr(&sh.empty[stage]), phase ^ 1, abort_flag, a.wait)) break;
        ptx::mbar_arrive_expect_tx(bar, a_bytes + b_bytes);
#pragma unroll
        for (int c = 0; c < BN / 64; ++c) {
          const uint32_t to = ptx::smem_addr(s_b + stage * b_bytes + c * (kBK * 128));
          if constexpr (G) ptx::tma_load_3d(to, &tmap_w, bar, col0 + c * 64, kb * kBK, group);
          else ptx::tma_load_2d(to, &tmap_w, bar, col0 + c * 64, kb * kBK);
        }
        ptx::tma_load_2d(ptx::smem_addr(s_a + stage * a_bytes), &tmap_x, bar, kb * kBK, row_load);
        ++fills;
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32(kSplitRows, BN, false, true);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        // everything but the MMAs is worked out before the wait, as the operands arrive just in time
        const int done_kb = kb - kb0, stretch = done_kb / kStretch;
        const bool first = kFine ? done_kb % kStretch == 0 : done_kb == 0;
        const uint32_t acc = kFine ? sh.tmem_base + (stretch & 1) * BN : sh.tmem_base;
        const uint64_t ad = ptx::sw128_desc(ptx::smem_addr(s_a + stage * a_bytes), 16, 1024);
        const uint64_t bd = ptx::sw128_desc(ptx::smem_addr(s_b + stage * b_bytes), kBK * 128, 1024);
        if (kFine && first && stretch >= 2 &&
            !ptx::mbar_wait_bounded(ptx::smem_addr(&sh.tempty[stretch & 1]), ((stretch >> 1) - 1) & 1, abort_flag,
                                    a.wait))
          break;
        if (!ptx::mbar_wait_bounded(ptx::smem_addr(&sh.full[stage]), phase, abort_flag, a.wait)) break;
        ptx::tc_fence_after();
        // the descriptors' address field counts 16 bytes: a step of 16 along k is 32 bytes of x and 16 rows of w
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          ptx::tc_mma_bf16(acc, ad + kk * 2, bd + kk * 128, idesc, (!first || kk > 0) ? 1u : 0u);
        ptx::tc_commit(ptx::smem_addr(&sh.empty[stage]));
        if (kFine && (kb == kb1 - 1 || done_kb % kStretch == kStretch - 1))
          ptx::tc_commit(ptx::smem_addr(&sh.tfull[stretch & 1]));
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // arrives when every MMA issued above is complete, after a wait that ran out too
      ptx::tc_commit(ptx::smem_addr(&sh.done));
    }
    __syncwarp();
  } else if (live) {
    // Warps 2 and 3, with bf16 outputs 4 to 7 too, have nothing to do until the sums are there: the tile's bias and this
    // CTA's rows of the residual to L2, a line each (the bias' few lines from one thread only: they are everybody's).
    constexpr int kLine = 128 / static_cast<int>(sizeof(O)), kLines = BN / kLine;
    constexpr int kIdle = kFine ? 64 : kSplitThreads - 64;
    const int i0 = static_cast<int>(threadIdx.x) - 64;
    if (bias_row != nullptr && i0 < BN / 32 && col0 + i0 * 32 < a.n) ptx::prefetch_l2(bias_row + col0 + i0 * 32);
    if (a.residual != nullptr && i0 < kIdle) {
      for (int i = i0 + rank * kIdle; i < (row_end - row0) * kLines; i += C * kIdle) {
        const int32_t col = col0 + (i % kLines) * kLine;
        if (col < a.n)
          ptx::prefetch_l2(static_cast<const O*>(a.residual) + static_cast<int64_t>(row0 + i / kLines) * a.n + col);
      }
    }
    __syncwarp();
  }
  if (G && (warp == 2 || warp == 3)) {
    const int thread = static_cast<int>(threadIdx.x) - 64;
    zero_rows(sh, L, a.out, static_cast<int64_t>(a.n) * static_cast<int64_t>(sizeof(O)), thread);
    if (a.pre != nullptr) zero_rows(sh, L, a.pre, static_cast<int64_t>(a.n) * 2, thread);
    __syncwarp();
  }
  if (kFine && warp >= 4) {
    // f32 outputs: each stretch of k is added to the row's sums in registers, with rounding
#pragma unroll
    for (int i = 0; i < (kFine ? BN : 1); ++i) sums[i] = 0.0f;
    const int stretches = (kb1 - kb0 + kStretch - 1) / kStretch;
#pragma unroll 1
    for (int s = 0; s < stretches; ++s) {
      bool there = ptx::mbar_wait_bounded(ptx::smem_addr(&sh.tfull[s & 1]), (s >> 1) & 1, abort_flag, a.wait);
      there = __all_sync(0xFFFFFFFFu, there);
      if (!there) break;
      ptx::tc_fence_after();
      const uint32_t from = sh.tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (s & 1) * BN;
#pragma unroll
      for (int c = 0; c < (kFine ? BN / 32 : 0); ++c) {
        uint32_t v[32];
        ptx::tmem_load_32cols(from + c * 32, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) sums[c * 32 + i] += __uint_as_float(v[i]);
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&sh.tempty[s & 1]));
    }
    __syncwarp();
  }
  {
    volatile int no_abort = 0;
    // (twice the bound of the other waits, which end first)
    if (!ptx::mbar_wait_bounded(ptx::smem_addr(&sh.done), 0, &no_abort, WaitBound{2 * a.wait.ns + kSplitDrain.ns, kSuspendHintNs})) *abort_flag = 1;
    // After a wait that ran out, whichever role's it was, the copies that no MMA has waited for land before the ring's place
    // is taken.  (The role may give up after the last copy has been asked for, so it is here that the flag is looked at: the
    // issuing thread raises it before the commit that ends this wait.)
    if (fills > 0 && *abort_flag) {
      const int last = fills < a.stages ? fills : a.stages;
      for (int i = 1; i <= last; ++i) {
        const int f = fills - i;
        ptx::mbar_wait_bounded(ptx::smem_addr(&sh.full[f % a.stages]), (f / a.stages) & 1, &no_abort, kSplitDrain);
      }
    }
    __syncwarp();
  }
  __syncthreads();  // every warp is past its waits: the ring is free, and all see the same flag
  const bool ok = *abort_flag == 0;
  ptx::tc_fence_after();

  // the accumulator's rows to shared memory: a thread a row, two warps a quarter of the rows
  float* stage_f = reinterpret_cast<float*>(smem);
  const int quarter = warp & 3;  // of tensor memory's lanes, the one that this warp may read
  const int tile_row = quarter * 32 + lane;
  if (kFine) {
    if (live && warp >= 4 && quarter * 32 < a.box_rows) {
      float4* dst = reinterpret_cast<float4*>(stage_f + tile_row * kPitch);
#pragma unroll
      for (int i = 0; i < (kFine ? BN / 4 : 0); ++i)
        dst[i] = make_float4(sums[4 * i], sums[4 * i + 1], sums[4 * i + 2], sums[4 * i + 3]);
    }
  } else if (live && quarter * 32 < a.box_rows) {
    const uint32_t tb = sh.tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
    for (int c = warp >> 2; c < BN / 32; c += kSplitThreads / 128) {
      uint32_t v[32];
      if (kb1 > kb0) {
        ptx::tmem_load_32cols(tb + c * 32, v);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0u;
      }
      float4* dst = reinterpret_cast<float4*>(stage_f + tile_row * kPitch + c * 32);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        dst[i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                             __uint_as_float(v[4 * i + 3]));
    }
  }
  ptx::tc_fence_before();
  if (C > 1) ptx::cluster_sync();
  else __syncthreads();

  // Every CTA of the cluster adds its share of the tile, its own sums first, then the others' in their order, in
  // units of four columns and batches whose loads (the units' sums from the other CTAs, bias and residual)
  // are all in flight at once: a remote load takes half a microsecond.  After its last remote loads it arrives at
  // the barrier that keeps the CTAs' shared memory until all have read it.
  constexpr int kBatch = C == 8 ? 2 : 4;  // units (more of them make code that is slower to fetch than the loads to wait for)
  constexpr int kUnits = BN / 4;                         // of a row
  const int32_t shift = row0 - row_load;                 // tile row of row0
  const int units = live && ok ? (row_end - row0) * kUnits : 0;
  const uint32_t base = ptx::smem_addr(stage_f);
  const O* residual = static_cast<const O*>(a.residual);
  O* out = static_cast<O*>(a.out);
  constexpr int kStride = C * kSplitThreads;
  bool arrived = C == 1;
  for (int first = 0; first < units || !arrived; first += kBatch * kStride) {
    const int u0 = first + rank * kSplitThreads + static_cast<int>(threadIdx.x);
    float4 part[kBatch][C > 1 ? C - 1 : 1], bias[kBatch];
    typename Quad<O>::Raw res[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = u0 + i * kStride, r = u / kUnits, c = (u % kUnits) * 4;
      if (u < units && col0 + c < a.n) {
        const uint32_t at = base + static_cast<uint32_t>(((r + shift) * kPitch + c) * 4);
#pragma unroll
        for (int s = 1; s < C; ++s) part[i][s - 1] = ld_cluster(ptx::map_to_rank(at, (rank + s) % C));
        if (bias_row != nullptr) bias[i] = *reinterpret_cast<const float4*>(bias_row + col0 + c);
        if (residual != nullptr)
          res[i] = *reinterpret_cast<const typename Quad<O>::Raw*>(
              residual + static_cast<int64_t>(row0 + r) * a.n + col0 + c);
      }
    }
    if (C > 1 && !arrived && first + kBatch * kStride >= units) {
      // the same batch for every thread of the block; the arrival orders this thread's loads before it
      __syncwarp();
      ptx::cluster_arrive();
      arrived = true;
    }
    with_act(a.act, [&](auto tag) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int u = u0 + i * kStride, r = u / kUnits, c = (u % kUnits) * 4;
        if (u >= units || col0 + c >= a.n) continue;
        float2 z[2];
        widen(*reinterpret_cast<const float4*>(stage_f + (r + shift) * kPitch + c), z);
#pragma unroll
        for (int s = 1; s < C; ++s) {
          z[0] = add2(z[0], make_float2(part[i][s - 1].x, part[i][s - 1].y));
          z[1] = add2(z[1], make_float2(part[i][s - 1].z, part[i][s - 1].w));
        }
        if (bias_row != nullptr) {
          z[0] = add2(z[0], make_float2(bias[i].x, bias[i].y));
          z[1] = add2(z[1], make_float2(bias[i].z, bias[i].w));
        }
        const int64_t place = static_cast<int64_t>(row0 + r) * a.n + col0 + c;
        if (a.pre != nullptr) store4(static_cast<bf16*>(a.pre) + place, z);
        z[0] = act_value<decltype(tag)::value>(z[0]);
        z[1] = act_value<decltype(tag)::value>(z[1]);
        if (residual != nullptr) {
          float2 e[2];
          widen(res[i], e);
          z[0] = add2(z[0], e[0]);
          z[1] = add2(z[1], e[1]);
        }
        store4(out + place, z);
      }
    });
  }
  __syncwarp();
  if (C > 1) ptx::cluster_wait();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(sh.tmem_base, kTmem);
  }
  if (threadIdx.x == 0 && !ok && a.status != nullptr) atomicOr(a.status, RD_STATUS_TIMEOUT);
}

template <class O, int BN, int C, bool G>
cudaError_t go(const CUtensorMap& tx, const CUtensorMap& tw, const SplitArgs& a, cudaStream_t stream) {
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(gemm_split_kernel<O, BN, C, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(split_smem(kSplitRingAlone)));
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  const dim3 grid(static_cast<unsigned>(ceil_div(a.n, BN)) * static_cast<unsigned>(C),
                  static_cast<unsigned>(a.row_tiles));
  return launch_pdl(gemm_split_kernel<O, BN, C, G>, grid, kSplitThreads, split_smem(a.ring_bytes), C, stream, tx, tw, a);
}

template <class O, int BN, bool G>
cudaError_t by_cluster(const CUtensorMap& tx, const CUtensorMap& tw, const SplitArgs& a, cudaStream_t stream) {
  if constexpr (BN == 128) return go<O, BN, 1, G>(tx, tw, a, stream);  // (tiles of 128 columns are enough for the SMs)
  else switch (a.cluster) {
    case 8: return go<O, BN, 8, G>(tx, tw, a, stream);
    case 4: return go<O, BN, 4, G>(tx, tw, a, stream);
    case 2: return go<O, BN, 2, G>(tx, tw, a, stream);
    default: return go<O, BN, 1, G>(tx, tw, a, stream);
  }
}

template <class O, bool G>
cudaError_t by_cols(int cols, const CUtensorMap& tx, const CUtensorMap& tw, const SplitArgs& a, cudaStream_t stream) {
  return cols == 64 ? by_cluster<O, 64, G>(tx, tw, a, stream) : by_cluster<O, 128, G>(tx, tw, a, stream);
}

}  // namespace

cudaError_t launch_gemm_split(bool f32_out, int cols, const CUtensorMap& tx, const CUtensorMap& tw,
                              const SplitArgs& a, cudaStream_t stream) {
  if (a.group_sizes == nullptr)
    return f32_out ? by_cols<float, false>(cols, tx, tw, a, stream) : by_cols<bf16, false>(cols, tx, tw, a, stream);
  return f32_out ? by_cols<float, true>(cols, tx, tw, a, stream) : by_cols<bf16, true>(cols, tx, tw, a, stream);
}

}  // namespace rd
