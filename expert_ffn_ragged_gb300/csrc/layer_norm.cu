// layer_norm.cu -- layer norm of rows and its gradients (rd_layer_norm_fwd, rd_layer_norm_bwd).
//
// Both directions are one pass over HBM.  T threads hold a row in registers, V quads of four elements each, so the
// mean, the squares about it and the result come from one read.  Blocks stay on the SM and take rows in turn:
// the next S - 1 rows are on their way to shared memory (cp.async, each thread into words that it alone reads,
// so no barrier is needed for them) while this row is summed.  A thread keeps the same columns throughout:
// weight and bias stay in registers, and the backward pass adds its columns' d_out * y and d_out there.
// At the end the blocks of a cluster add their two sums a column through distributed shared memory, in their
// order, and write one part a cluster to the workspace; a second kernel adds the parts in theirs (no atomics).  (Up to 1024 rows: below.)
// Rows of the backward pass too long for one block's registers (past 8192) are shared by a cluster, whose blocks send
// each other the row's two sums; past 65536 the row is read twice and the columns are summed by a kernel of their own.
//
// Bound: HBM.  28157 x 4096, f32 stream, bf16 in the products: forward 692 MB in 106 us (6.5 TB/s), gradients 1.15 GB in
// 175 us (6.6 TB/s, the second kernel's 3 us among them).  bf16 throughout the gradients take 121 us (5.7 TB/s): issue
// slots, 22 packed operations for four elements.  One row takes 2.0 us, 509 rows' gradients 6.3 us, in one launch (in the two
// of the many rows, each some 4 us from its start to its first result, 10.4).
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "act_math.cuh"
#include "block_args.h"
#include "launch.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace rd {
namespace {

// ------------------------------------------------------------------ forward
// T threads hold R rows of V quads a thread; a block of fewer than 128 such threads takes several row groups
template <int T>
struct Shape {
  static constexpr int kThreads = T == 32 ? 256 : T;
  static constexpr int kGroups = kThreads / T;
};

template <class X, class O, int T, int V, int R, int S, int B>
__global__ void __launch_bounds__(Shape<T>::kThreads, B) layer_norm_fwd_kernel(const NormArgs a) {
  constexpr int kThreads = Shape<T>::kThreads, kGroups = Shape<T>::kGroups;
  constexpr bool kHold = T <= 512;  // weight and bias in registers
  using Raw = typename Quad<X>::Raw;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float sums[32 * R];
  __shared__ __align__(16) float pairs[32 * 2 * R];
  pdl_trigger();
  pdl_wait();
  Raw* ring = reinterpret_cast<Raw*>(smem) + threadIdx.x;
  const int t = threadIdx.x % T;
  const int quads = a.hidden >> 2;
  const int64_t hidden = a.hidden;
  const int32_t L = rows_within(a.limit, a.rows);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups * R;
  const float inv = 1.0f / static_cast<float>(a.hidden);
  const X* x = static_cast<const X*>(a.x) + 4 * t;
  O* out = static_cast<O*>(a.out) + 4 * t;
  int64_t row = (static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / T) * R;
  if (row >= L) return;
  auto fetch = [&](int64_t first, int s) {
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (first + j < L) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (t + i * T < quads)
            quad_copy(ring + ((s * R + j) * V + i) * kThreads, x + (first + j) * hidden + 4 * i * T);
      }
    copies_commit();
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(row + s * step, s);
  auto param = [&](const float* p, int i, float none, float2 (&v)[2]) {
    if (p != nullptr) {
      widen(*reinterpret_cast<const float4*>(p + 4 * (t + i * T)), v);
    } else {
      v[0] = v[1] = both(none);
    }
  };
  float2 w[kHold ? V : 1][2], b[kHold ? V : 1][2];
  if (kHold) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < quads) {
        param(a.weight, i, 1.0f, w[i]);
        param(a.bias, i, 0.0f, b[i]);
      }
  }
  int stage = 0;
  for (; row < L; row += step) {
    fetch(row + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
    copies_wait<S - 1>();
    // rows past the last one hold whatever the ring held: their sums are not used
    float2 v[R][V][2];
    float mean[R], cq[2 * R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float2 s2 = both(0.0f);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (t + i * T < quads) {
          widen(ring[((stage * R + j) * V + i) * kThreads], v[j][i]);
          s2 = add2(s2, add2(v[j][i][0], v[j][i][1]));
        }
      mean[j] = s2.x + s2.y;
    }
    if (++stage == S) stage = 0;
    row_sums<T>(mean, sums);
    // What is left of the mean after its rounding (c) is taken out too: a row far from zero would
    // otherwise be off by an ulp of its mean.
#pragma unroll
    for (int j = 0; j < R; ++j) {
      mean[j] *= inv;
      float2 c2 = both(0.0f), q2 = both(0.0f);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (t + i * T < quads) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            v[j][i][e] = add2(v[j][i][e], both(-mean[j]));
            c2 = add2(c2, v[j][i][e]);
            q2 = fma2(v[j][i][e], v[j][i][e], q2);
          }
        }
      cq[2 * j] = c2.x + c2.y;
      cq[2 * j + 1] = q2.x + q2.y;
    }
    row_sums<T>(cq, pairs);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float c = cq[2 * j] * inv;
      const float var = fmaf(-c, c, cq[2 * j + 1] * inv);  // never below zero but by rounding; NaN stays NaN
      const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + a.eps);
      const float2 r2 = both(rstd), back = both(-c * rstd);
      if (R > 1 && row + j >= L) break;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (t + i * T < quads) {
          if (!kHold) {
            param(a.weight, i, 1.0f, w[0]);
            param(a.bias, i, 0.0f, b[0]);
          }
          const int h = kHold ? i : 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) v[j][i][e] = fma2(fma2(v[j][i][e], r2, back), w[h][e], b[h][e]);
          store4(out + (row + j) * hidden + 4 * i * T, v[j][i]);
        }
      if (t == 0 && a.mean != nullptr) {
        a.mean[row + j] = mean[j] + c;
        a.rstd[row + j] = rstd;
      }
    }
  }
}

// rows too long for registers: three reads of the row, of which the last two come from L2
template <class X, class O>
__global__ void __launch_bounds__(1024) layer_norm_fwd_long_kernel(const NormArgs a) {
  __shared__ __align__(16) float sums[32];
  __shared__ __align__(16) float pairs[64];
  pdl_trigger();
  pdl_wait();
  const int vecs = a.hidden >> 3;
  const int64_t hidden = a.hidden;
  const int32_t L = rows_within(a.limit, a.rows);
  const float inv = 1.0f / static_cast<float>(a.hidden);
  for (int64_t row = blockIdx.x; row < L; row += gridDim.x) {
    const X* x = static_cast<const X*>(a.x) + row * hidden;
    O* out = static_cast<O*>(a.out) + row * hidden;
    float s[1] = {0.0f}, cq[2] = {0.0f, 0.0f};
    for (int64_t v = threadIdx.x; v < vecs; v += 1024) {
      float e[8];
      load8(x + 8 * v, e);
      s[0] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    }
    row_sums<1024>(s, sums);
    const float mean = s[0] * inv;
    for (int64_t v = threadIdx.x; v < vecs; v += 1024) {
      float e[8];
      load8(x + 8 * v, e);
      float k = 0.0f, p = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        k += e[i] - mean;
        p = fmaf(e[i] - mean, e[i] - mean, p);
      }
      cq[0] += k;
      cq[1] += p;
    }
    row_sums<1024>(cq, pairs);
    const float c = cq[0] * inv;
    const float var = fmaf(-c, c, cq[1] * inv);  // never below zero but by rounding; NaN stays NaN
    const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + a.eps);
    for (int64_t v = threadIdx.x; v < vecs; v += 1024) {
      float e[8], w[8], b[8];
      load8(x + 8 * v, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.0f, b[i] = 0.0f;
      if (a.weight != nullptr) load8_param(a.weight + 8 * v, w);
      if (a.bias != nullptr) load8_param(a.bias + 8 * v, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = fmaf((e[i] - mean - c) * rstd, w[i], b[i]);
      store8(out + 8 * v, e);
    }
    if (threadIdx.x == 0 && a.mean != nullptr) {
      a.mean[row] = mean + c;
      a.rstd[row] = rstd;
    }
  }
}

// ------------------------------------------------------------------ backward
constexpr int kNormCluster = 2;  // blocks that add their sums before they go to the workspace

constexpr int kNormMaxSplit = 8;  // blocks that share a row too long for one
constexpr uint64_t kNormGraceNs = 200000ull;  // for sums on their way to a block that no longer waits for them

// two sums to the same words of another block of the cluster, counted on its barrier there (no fence: a release at
// cluster scope would wait for the row's global stores too)
__device__ __forceinline__ void put_peer(float2* local, uint64_t* bar, int rank, float x, float y) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                   ptx::map_to_rank(ptx::smem_addr(local), static_cast<uint32_t>(rank))),
               "f"(x), "f"(y), "r"(ptx::map_to_rank(ptx::smem_addr(bar), static_cast<uint32_t>(rank)))
               : "memory");
}

__device__ __forceinline__ float4 peer_float4(const float4* local, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(ptx::map_to_rank(ptx::smem_addr(local), static_cast<uint32_t>(rank)))
               : "memory");
  return v;
}

// A bounded wait for the other blocks' sums.  Its tries have their usual window whatever the bound: a window read from the
// arguments costs 1 % of the kernel's time (1760 x 65536 in bf16 190.6 us instead of 188.4).
__device__ __forceinline__ bool wait_for_sums(uint32_t bar, uint32_t parity, volatile int* gave_up, uint64_t limit_ns) {
  if (ptx::mbar_try_wait_cluster(bar, parity, kSuspendHintNs)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
#pragma unroll 1
  while (true) {
    if (ptx::mbar_try_wait_cluster(bar, parity, kSuspendHintNs)) return true;
    if (*gave_up) return false;
    if (ptx::global_timer_ns() - t0 > limit_ns) {
      *gave_up = 1;
      return false;
    }
  }
}

// SPLIT: a cluster holds a row, each block split_cols (at most kCols) of its columns; the row's two sums cross the cluster
template <class X, class O, int T, int V, int R, int S, int B, bool SPLIT>
__global__ void __launch_bounds__(Shape<T>::kThreads, B) layer_norm_bwd_kernel(const NormArgs a) {
  constexpr int kThreads = Shape<T>::kThreads, kGroups = Shape<T>::kGroups;
  constexpr int kCols = T * V * 4;
  using RawX = typename Quad<X>::Raw;
  using RawO = typename Quad<O>::Raw;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float pairs[2][32 * 2 * R];
  __shared__ float2 joined[2][kNormMaxSplit][R];  // SPLIT: the sums of the cluster's blocks
  __shared__ uint64_t joined_full[2];
  __shared__ int gave_up;
  static_assert(!SPLIT || T != 32, "a block's threads share their rows");
  if (SPLIT) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < 2; ++i) ptx::mbar_init(ptx::smem_addr(&joined_full[i]), 1);
      gave_up = 0;
      ptx::fence_mbar_init();
    }
    ptx::cluster_sync();  // every block of the cluster runs and its barriers are ready
  }
  pdl_trigger();
  pdl_wait();
  const int split = SPLIT ? a.split : 1;
  const int rank = SPLIT ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int64_t col0 = SPLIT ? static_cast<int64_t>(rank) * a.split_cols : 0;  // of this block
  RawX* ring_x = reinterpret_cast<RawX*>(smem) + threadIdx.x;
  RawO* ring_d = reinterpret_cast<RawO*>(smem + S * R * V * kThreads * sizeof(RawX)) + threadIdx.x;
  const int t = threadIdx.x % T;
  const int64_t cols = SPLIT && a.hidden - col0 > a.split_cols ? a.split_cols : a.hidden - col0;
  const int quads = static_cast<int>(cols >> 2);
  const int64_t hidden = a.hidden;
  const int32_t L = rows_within(a.limit, a.rows);
  const int blocks = SPLIT ? gridDim.x / split : gridDim.x;  // (clusters)
  const int block = SPLIT ? blockIdx.x / split : blockIdx.x;
  const int64_t step = static_cast<int64_t>(blocks) * kGroups * R;
  const float inv = 1.0f / static_cast<float>(a.hidden);
  const X* x = static_cast<const X*>(a.x) + col0 + 4 * t;
  const O* d_out = static_cast<const O*>(a.d_out) + col0 + 4 * t;
  X* d_x = static_cast<X*>(a.out) + col0 + 4 * t;
  const float* weight = a.weight == nullptr ? nullptr : a.weight + col0;
  int64_t row = (static_cast<int64_t>(block) * kGroups + threadIdx.x / T) * R;
  auto fetch = [&](int64_t first, int s) {
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (first + j < L) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (t + i * T < quads) {
            quad_copy(ring_x + ((s * R + j) * V + i) * kThreads, x + (first + j) * hidden + 4 * i * T);
            quad_copy(ring_d + ((s * R + j) * V + i) * kThreads, d_out + (first + j) * hidden + 4 * i * T);
          }
      }
    copies_commit();
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(row + s * step, s);
  float2 w[V][2], dw[V][2], db[V][2];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w[i][0] = w[i][1] = both(1.0f);
    dw[i][0] = dw[i][1] = db[i][0] = db[i][1] = both(0.0f);
    if (weight != nullptr && t + i * T < quads)
      widen(*reinterpret_cast<const float4*>(weight + 4 * (t + i * T)), w[i]);
  }
  float mean_next[R], rstd_next[R];
  auto stats = [&](int64_t first) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      mean_next[j] = rstd_next[j] = 0.0f;
      if (first + j < L) {
        mean_next[j] = a.mean[first + j];
        rstd_next[j] = a.rstd[first + j];
      }
    }
  };
  stats(row);
  uint32_t joined_phase = 0;  // a bit a slot
  // SPLIT: no wait of this thread has run out.  Sums cross a cluster within the window of a try, so with a bound below that
  // the first block starts as one that has given up, and the others' waits for its sums run out.
  bool there = rank != 0 || a.wait.try_ns == kSuspendHintNs;
  int stage = 0, slot = 0;
  for (; row < L; row += step) {
    fetch(row + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
    float2 r2[R], m2[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      r2[j] = both(rstd_next[j]);
      m2[j] = both(-mean_next[j]);
    }
    stats(row + step);
    copies_wait<S - 1>();
    float2 y[R][V][2], d[R][V][2];
    float pq[2 * R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float2 p2 = both(0.0f), q2 = both(0.0f);
      if (R == 1 || row + j < L) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (t + i * T < quads) {
            widen(ring_x[((stage * R + j) * V + i) * kThreads], y[j][i]);
            widen(ring_d[((stage * R + j) * V + i) * kThreads], d[j][i]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y[j][i][e] = mul2(add2(y[j][i][e], m2[j]), r2[j]);
              dw[i][e] = fma2(d[j][i][e], y[j][i][e], dw[i][e]);
              db[i][e] = add2(db[i][e], d[j][i][e]);
              d[j][i][e] = mul2(d[j][i][e], w[i][e]);
              p2 = add2(p2, d[j][i][e]);
              q2 = fma2(d[j][i][e], y[j][i][e], q2);
            }
          }
      }
      pq[2 * j] = p2.x + p2.y;
      pq[2 * j + 1] = q2.x + q2.y;
    }
    if (++stage == S) stage = 0;
    row_sums<T>(pq, pairs[slot]);
    if (SPLIT) {
      // Every block's sums to every block.  A slot's words are written again two turns on, by threads that have seen this
      // block's sums of the turn in between, which it sends after it has read the slot.  A thread whose wait has run
      // out sends no more (it does not know that the others have read theirs): their waits then run out too, and no
      // element gets another row's sums.
      const uint32_t bar = ptx::smem_addr(&joined_full[slot]);
      if (threadIdx.x == 0 && there) ptx::mbar_arrive_expect_tx(bar, split * R * 8);
      if (threadIdx.x < split && there) {
#pragma unroll
        for (int j = 0; j < R; ++j)
          put_peer(&joined[slot][rank][j], &joined_full[slot], static_cast<int>(threadIdx.x), pq[2 * j], pq[2 * j + 1]);
      }
      there = wait_for_sums(bar, (joined_phase >> slot) & 1u, &gave_up, a.wait.ns) && there;
      joined_phase ^= 1u << slot;
#pragma unroll
      for (int j = 0; j < 2 * R; ++j) pq[j] = 0.0f;
      for (int i = 0; i < split; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) {
          pq[2 * j] += joined[slot][i][j].x;
          pq[2 * j + 1] += joined[slot][i][j].y;
        }
      if (!there) {
        // a block of the cluster did not come in time: this row and the ones after it show it
#pragma unroll
        for (int j = 0; j < 2 * R; ++j) pq[j] = __int_as_float(0x7FC00000);
      }
    }
    slot ^= 1;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (R > 1 && row + j >= L) break;
      // d_x = rstd g - rstd p / h - y rstd q / h
      const float2 p2 = both(-pq[2 * j] * inv * r2[j].x), q2 = both(-pq[2 * j + 1] * inv * r2[j].x);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (t + i * T < quads) {
#pragma unroll
          for (int e = 0; e < 2; ++e) d[j][i][e] = fma2(y[j][i][e], q2, fma2(d[j][i][e], r2[j], p2));
          store4(d_x + (row + j) * hidden + 4 * i * T, d[j][i]);
        }
    }
  }
  if (SPLIT) {
    // Every block has sent its last sums, and has those sent to it, unless one of its waits ran out: then some may still be
    // on their way to its shared memory.
    ptx::cluster_sync();
    if (*static_cast<volatile int*>(&gave_up)) {
      const uint64_t t0 = ptx::global_timer_ns();
      while (ptx::global_timer_ns() - t0 < kNormGraceNs) __nanosleep(1000);
    }
    if (a.parts == nullptr) return;
    float* part = a.parts + static_cast<int64_t>(block) * 2 * hidden + col0 + 4 * t;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < quads) {
        store4(part + 4 * i * T, dw[i]);
        store4(part + hidden + 4 * i * T, db[i]);
      }
    return;
  }
  if (a.parts == nullptr) return;  // the same in every block
  // the ring's place is taken by this block's sums: [rows of the block][d_weight, d_bias][columns]
  copies_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float* at = sums + (threadIdx.x / T) * 2 * kCols + 4 * (t + i * T);
    store4(at, dw[i]);
    store4(at + kCols, db[i]);
  }
  ptx::cluster_sync();
  const int peer = static_cast<int>(ptx::cluster_ctarank());
  float* part = a.parts + static_cast<int64_t>(blockIdx.x / kNormCluster) * 2 * hidden;
  for (int u = peer * kThreads + threadIdx.x; u < kCols / 2; u += kNormCluster * kThreads) {
    const int k = u / (kCols / 4), quad = u - k * (kCols / 4);
    if (quad >= quads) continue;
    float2 s[2] = {both(0.0f), both(0.0f)};
#pragma unroll
    for (int c = 0; c < kNormCluster; ++c)
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const float4 v = peer_float4(reinterpret_cast<const float4*>(sums + (i * 2 + k) * kCols) + quad, c);
        s[0] = add2(s[0], make_float2(v.x, v.y));
        s[1] = add2(s[1], make_float2(v.z, v.w));
      }
    store4(part + k * hidden + 4 * quad, s);
  }
  ptx::cluster_sync();  // no block leaves while another reads its sums
}

// rows too long for registers: d_x alone, the row read twice (the second time from L2)
template <class X, class O>
__global__ void __launch_bounds__(1024) layer_norm_dx_long_kernel(const NormArgs a) {
  __shared__ __align__(16) float slots[2][64];
  pdl_trigger();
  pdl_wait();
  const int vecs = a.hidden >> 3;
  const int64_t hidden = a.hidden;
  const int32_t L = rows_within(a.limit, a.rows);
  const float inv = 1.0f / static_cast<float>(a.hidden);
  int slot = 0;
  for (int64_t row = blockIdx.x; row < L; row += gridDim.x, slot ^= 1) {
    const X* x = static_cast<const X*>(a.x) + row * hidden;
    const O* d_out = static_cast<const O*>(a.d_out) + row * hidden;
    X* d_x = static_cast<X*>(a.out) + row * hidden;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float pq[2] = {0.0f, 0.0f};
    auto at = [&](int64_t v, float (&y)[8], float (&d)[8]) {
      load8(x + 8 * v, y);
      load8(d_out + 8 * v, d);
      if (a.weight != nullptr) {
        float w[8];
        load8_param(a.weight + 8 * v, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = (y[i] - mean) * rstd;
    };
    for (int64_t v = threadIdx.x; v < vecs; v += 1024) {
      float y[8], d[8], pv = 0.0f, qv = 0.0f;
      at(v, y, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pv += d[i];
        qv = fmaf(d[i], y[i], qv);
      }
      pq[0] += pv;
      pq[1] += qv;
    }
    row_sums<1024>(pq, slots[slot]);
    const float p = pq[0] * inv, q = pq[1] * inv;
    for (int64_t v = threadIdx.x; v < vecs; v += 1024) {
      float y[8], d[8];
      at(v, y, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = rstd * (d[i] - fmaf(y[i], q, p));
      store8(d_x + 8 * v, d);
    }
  }
}

// ... and their columns' sums over a chunk of rows: 256 columns a block, eight rows at a time
template <class X, class O>
__global__ void __launch_bounds__(256) layer_norm_columns_kernel(const NormArgs a, int32_t chunk_rows) {
  __shared__ float across[8][2][256];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t hidden = a.hidden;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + lane * 8;
  const int32_t L = rows_within(a.limit, a.rows);
  const int64_t lo = static_cast<int64_t>(blockIdx.y) * chunk_rows;
  const int64_t hi = lo + chunk_rows < L ? lo + chunk_rows : L;
  float dw[8], db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.0f;
  if (col < hidden) {
#pragma unroll 4
    for (int64_t row = lo + warp; row < hi; row += 8) {
      float y[8], d[8];
      load8(static_cast<const X*>(a.x) + row * hidden + col, y);
      load8(static_cast<const O*>(a.d_out) + row * hidden + col, d);
      const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[i] = fmaf(d[i], (y[i] - mean) * rstd, dw[i]);
        db[i] += d[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    across[warp][0][lane * 8 + i] = dw[i];
    across[warp][1][lane * 8 + i] = db[i];
  }
  __syncthreads();
  float* part = a.parts + static_cast<int64_t>(blockIdx.y) * 2 * hidden;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= hidden) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += across[i][k][threadIdx.x];
    part[k * hidden + c] = s;
  }
}

// The parts to the gradients: 32 columns a block, sixteen threads a column, each every sixteenth part in
// order (few enough loads to be in flight at once).
constexpr int kPartLanes = 16;
__global__ void __launch_bounds__(32 * kPartLanes) layer_norm_parts_kernel(const NormArgs a, int32_t parts) {
  __shared__ float across[kPartLanes][33];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cols = 2 * static_cast<int64_t>(a.hidden);
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < cols) {
    const float* p = a.parts + c;
#pragma unroll 10
    for (int i = warp; i < parts; i += kPartLanes) s += p[i * cols];
  }
  across[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= cols) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < kPartLanes; ++i) s += across[i][lane];
  float* out = c < a.hidden ? a.d_weight : a.d_bias;
  if (out != nullptr) out[c < a.hidden ? c : c - a.hidden] = s;
}

// Few rows: everything in one launch and no workspace.  The first blocks take 32 columns each and read all rows for their sums
// (64 rows at a time, in a fixed order), the others a row a block (T = 256) or a warp (T = 32) for d_x; what both read comes
// from HBM once and from L2 once.
template <class X, class O, int T, int V>
__global__ void __launch_bounds__(256) layer_norm_bwd_few_kernel(const NormArgs a, int32_t col_blocks) {
  __shared__ __align__(16) float pairs[8 * 2];
  __shared__ float across[8][2][32];
  pdl_trigger();
  pdl_wait();
  const int64_t hidden = a.hidden;
  const int32_t L = rows_within(a.limit, a.rows);
  const X* x = static_cast<const X*>(a.x);
  const O* d_out = static_cast<const O*>(a.d_out);
  if (static_cast<int32_t>(blockIdx.x) < col_blocks) {
    const int piece = threadIdx.x & 3, row_lane = threadIdx.x >> 2, warp = threadIdx.x >> 5;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 32, col = col0 + piece * 8;
    float2 dw[4], db[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[i] = db[i] = both(0.0f);
    if (col < hidden) {
#pragma unroll 4
      for (int32_t row = row_lane; row < L; row += 64) {
        float y[8], d[8];
        load8(x + row * hidden + col, y);
        load8(d_out + row * hidden + col, d);
        const float2 m2 = both(-a.mean[row]), r2 = both(a.rstd[row]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 d2 = make_float2(d[2 * i], d[2 * i + 1]);
          dw[i] = fma2(d2, mul2(add2(make_float2(y[2 * i], y[2 * i + 1]), m2), r2), dw[i]);
          db[i] = add2(db[i], d2);
        }
      }
    }
#pragma unroll
    for (int s = 4; s < 32; s <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dw[i].x += __shfl_xor_sync(0xFFFFFFFFu, dw[i].x, s);
        dw[i].y += __shfl_xor_sync(0xFFFFFFFFu, dw[i].y, s);
        db[i].x += __shfl_xor_sync(0xFFFFFFFFu, db[i].x, s);
        db[i].y += __shfl_xor_sync(0xFFFFFFFFu, db[i].y, s);
      }
    if ((threadIdx.x & 31) < 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        across[warp][0][piece * 8 + 2 * i] = dw[i].x;
        across[warp][0][piece * 8 + 2 * i + 1] = dw[i].y;
        across[warp][1][piece * 8 + 2 * i] = db[i].x;
        across[warp][1][piece * 8 + 2 * i + 1] = db[i].y;
      }
    }
    __syncthreads();
    if (threadIdx.x >= 64) return;
    const int c = threadIdx.x & 31, which = threadIdx.x >> 5;
    float* out = which == 0 ? a.d_weight : a.d_bias;
    if (out == nullptr || col0 + c >= hidden) return;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += across[i][which][c];
    out[col0 + c] = s;
    return;
  }
  const int64_t row = (static_cast<int64_t>(blockIdx.x) - col_blocks) * (256 / T) + threadIdx.x / T;
  if (row >= L) return;
  const int t = threadIdx.x % T, vecs = a.hidden >> 3;
  const float inv = 1.0f / static_cast<float>(a.hidden), mean = a.mean[row], rstd = a.rstd[row];
  float y[V][8], d[V][8], pq[2] = {0.0f, 0.0f};
  Raw8<X> rx[V];
  Raw8<O> rd[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (t + i * T < vecs) {
      load_raw(rx[i], x + row * hidden + 8 * (t + i * T));
      load_raw(rd[i], d_out + row * hidden + 8 * (t + i * T));
    }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (t + i * T < vecs) {
      float w[8];
      widen(rx[i], y[i]);
      widen(rd[i], d[i]);
      if (a.weight != nullptr) {
        load8_param(a.weight + 8 * (t + i * T), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[i][e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[i][e] = (y[i][e] - mean) * rstd;
        pq[0] += d[i][e];
        pq[1] = fmaf(d[i][e], y[i][e], pq[1]);
      }
    }
  row_sums<T>(pq, pairs);
  const float p = pq[0] * inv, q = pq[1] * inv;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (t + i * T < vecs) {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[i][e] = rstd * (d[i][e] - fmaf(y[i][e], q, p));
      store8(static_cast<X*>(a.out) + row * hidden + 8 * (t + i * T), d[i]);
    }
}

int64_t ceil_of(int64_t n, int64_t d) { return (n + d - 1) / d; }


template <class X, class O, int T, int V>
cudaError_t bwd_few(const NormArgs& a, cudaStream_t stream) {
  const bool sums = a.d_weight != nullptr || a.d_bias != nullptr;
  const int64_t cols = sums ? ceil_of(a.hidden, 32) : 0, blocks = cols + ceil_of(a.rows, 256 / T);
  return launch_pdl(layer_norm_bwd_few_kernel<X, O, T, V>, dim3(static_cast<unsigned>(blocks)), 256, 0, 1, stream, a,
                    static_cast<int32_t>(cols));
}

template <class X, class O>
cudaError_t bwd_few_by_width(const NormArgs& a, cudaStream_t stream) {
  if (a.hidden <= 256) return bwd_few<X, O, 32, 1>(a, stream);
  if (a.hidden <= 1024) return bwd_few<X, O, 32, 4>(a, stream);
  if (a.hidden <= 4096) return bwd_few<X, O, 256, 2>(a, stream);
  return bwd_few<X, O, 256, 4>(a, stream);
}

// R rows at a time, S of these in the ring, B blocks on an SM
template <class X, class O, int T, int V, int R, int S, int B>
cudaError_t fwd(const NormArgs& a, int sms, cudaStream_t stream) {
  constexpr size_t smem = static_cast<size_t>(S) * R * V * Shape<T>::kThreads * sizeof(typename Quad<X>::Raw);
  auto* kernel = layer_norm_fwd_kernel<X, O, T, V, R, S, B>;
  static std::atomic<bool> set[64];
  int dev = 0;
  const cudaError_t e = allow_smem(kernel, smem, set, &dev);
  if (e != cudaSuccess) return e;
  const int64_t blocks = ceil_of(a.rows, Shape<T>::kGroups * R), most = static_cast<int64_t>(sms) * B;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), Shape<T>::kThreads, smem, 1,
                    stream, a);
}

template <class X, class O>
cudaError_t fwd_by_width(const NormArgs& a, int sms, cudaStream_t stream) {
  const int quads = a.hidden / 4;
  // Long pieces of a row a thread and few threads a row (little to exchange), and no more bytes on their way than it
  // takes: with 1024 threads an SM and three rows in the ring, 28157 x 4096 f32 took 122 us instead of 106.
  // GB/s of f32 to bf16 / bf16 to bf16 / f32 to f32, other forms in brackets:
  //   256:  - / 5300 / -   (one row at a time 4820, no fewer than three blocks)
  //   1024: - / 6020 / -   (64 x 4: 5560, 128 x 2 x 2 rows: 5010)
  //   2048: - / 6170 / -   (128 x 4: 5760)
  //   4096: 6540 / 6300 / 6630   (256 x 4: bf16 5750, f32 to f32 on three blocks 5810; 128 x 8: f32 6290)
  //   8192: 6270 / - / -   (512 x 4: 5790);  16384: 6480 / - / -   (1024 x 4: 4730)
  if (quads <= 64) return fwd<X, O, 32, 2, 2, 2, 3>(a, sms, stream);
  if (quads <= 128) return fwd<X, O, 32, 4, 1, 2, 3>(a, sms, stream);
  if (quads <= 256) return fwd<X, O, 32, 8, 1, 2, 2>(a, sms, stream);
  if (quads <= 512) return fwd<X, O, 64, 8, 1, 2, 8>(a, sms, stream);
  if (quads <= 1024) {
    if (sizeof(X) == 2) return fwd<X, O, 128, 8, 1, 2, 4>(a, sms, stream);
    return fwd<X, O, 256, 4, 1, 2, sizeof(O) == 4 ? 2 : 3>(a, sms, stream);
  }
  if (quads <= 2048) return fwd<X, O, 256, 8, 1, 2, 2>(a, sms, stream);
  if (quads <= 4096) return fwd<X, O, 512, 8, 1, 2, 1>(a, sms, stream);
  if (quads <= 8192) return fwd<X, O, 1024, 8, 1, 1, 1>(a, sms, stream);
  const int64_t most = 2 * static_cast<int64_t>(sms);
  return launch_pdl(layer_norm_fwd_long_kernel<X, O>, dim3(static_cast<unsigned>(a.rows < most ? a.rows : most)),
                    1024, 0, 1, stream, a);
}

// the backward kernel that holds rows in registers: rows that a block takes at a time, blocks on an SM and
// blocks that share a row; 0: rows are too long for it
struct BwdShape {
  int rows, blocks, split;
};
BwdShape bwd_shape(int64_t hidden) {
  if (hidden <= 256) return {8, 3, 1};
  if (hidden <= 1024) return {2, 4, 1};
  if (hidden <= 2048) return {2, 2, 1};
  if (hidden <= 4096) return {1, 2, 1};
  if (hidden <= 8192) return {1, 1, 1};
  // clusters of 2, 4 or 8, which leave few SMs without work (clusters of three took 190 or 277 us for 9385 x 12288, as 46 of
  // them, the most by the runtime's count, sometimes did not run at once)
  if (hidden <= 8192 * kNormMaxSplit) return {1, 1, hidden <= 16384 ? 2 : (hidden <= 32768 ? 4 : 8)};
  return {0, 0, 1};
}

template <class X, class O, int T, int V, int R, int B, bool SPLIT = false>
cudaError_t bwd(const NormArgs& a, int* parts, cudaStream_t stream) {
  constexpr int S = SPLIT ? 3 : 2;
  constexpr size_t ring = static_cast<size_t>(S) * R * V * Shape<T>::kThreads *
                          (sizeof(typename Quad<X>::Raw) + sizeof(typename Quad<O>::Raw));
  constexpr size_t sums = static_cast<size_t>(Shape<T>::kGroups) * 2 * T * V * 4 * 4;
  constexpr size_t smem = ring > sums ? ring : sums;
  auto* kernel = layer_norm_bwd_kernel<X, O, T, V, R, S, B, SPLIT>;
  const int cluster = SPLIT ? a.split : kNormCluster;
  static std::atomic<bool> set[64];
  static std::atomic<int> known[64][kNormMaxSplit + 1];  // clusters on the device at once, by their size
  int dev = 0;
  cudaError_t e = allow_smem(kernel, smem, set, &dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>& resident = known[dev][cluster];
  int clusters = resident.load(std::memory_order_acquire);
  if (clusters == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster), 1, 1);
    cfg.blockDim = dim3(Shape<T>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters < 1) clusters = 1;
    resident.store(clusters, std::memory_order_release);
  }
  if (clusters < *parts) *parts = clusters;
  // as few clusters as take the same number of turns: their parts are read again (when 509 x 4096 came this way: 10.8 us
  // with 152, 10.3 with 128)
  const int64_t units = ceil_of(a.rows, (SPLIT ? 1 : cluster) * Shape<T>::kGroups * R);
  if (units > 0) *parts = static_cast<int>(ceil_of(units, ceil_of(units, *parts)));
  return launch_pdl(kernel, dim3(static_cast<unsigned>(*parts * cluster)), Shape<T>::kThreads, smem, cluster, stream, a);
}

// GB/s with f32 rows and bf16 d_out / bf16 both, other forms in brackets:
//   256: - / 5110 (two rows at a time 3360);  1024: - / 5820 (64 threads x 4 quads 4650);  2048: - / 5670
//   4096: 6580 / 5710 (512 threads x 2 quads, two rows at a time: 6410 / 5070; one row: 5420 / 4350);  8192: 6530 / -
//   12288: - / 3860, 16384: 6070 / -, 32768: - / 4360 (two rows at a time over twice as many blocks 3630, 5570, 3050; a row
//   read twice by one block instead of shared by a cluster 1970, 2970, 2200)
template <class X, class O>
cudaError_t bwd_by_width(const NormArgs& a, int* parts, int sms, cudaStream_t stream) {
  if (layer_norm_bwd_few(a.rows, a.hidden)) return bwd_few_by_width<X, O>(a, stream);
  // (rows at a time and blocks as bwd_shape has them)
  if (a.hidden <= 256) return bwd<X, O, 32, 2, 1, 3>(a, parts, stream);
  if (a.hidden <= 1024) return bwd<X, O, 128, 2, 2, 4>(a, parts, stream);
  if (a.hidden <= 2048) return bwd<X, O, 256, 2, 2, 2>(a, parts, stream);
  if (a.hidden <= 4096) return bwd<X, O, 256, 4, 1, 2>(a, parts, stream);
  if (a.hidden <= 8192) return bwd<X, O, 512, 4, 1, 1>(a, parts, stream);
  const int split = bwd_shape(a.hidden).split;
  if (split > 1) {
    NormArgs shared = a;
    shared.split = split;
    shared.split_cols = static_cast<int32_t>(ceil_of(a.hidden, 64 * split) * 64);  // whole lines
    return bwd<X, O, 512, 4, 1, 1, true>(shared, parts, stream);
  }
  const int64_t most = 2 * static_cast<int64_t>(sms);
  if (a.rows > 0) {
    const cudaError_t e = launch_pdl(layer_norm_dx_long_kernel<X, O>,
                                     dim3(static_cast<unsigned>(a.rows < most ? a.rows : most)), 1024, 0, 1, stream, a);
    if (e != cudaSuccess) return e;
  }
  if (a.parts == nullptr) return cudaSuccess;
  return launch_pdl(layer_norm_columns_kernel<X, O>,
                    dim3(static_cast<unsigned>(ceil_of(a.hidden, 256)), static_cast<unsigned>(*parts)), 256, 0, 1,
                    stream, a, static_cast<int32_t>(ceil_of(a.rows, *parts)));
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const NormArgs& a, int dtype, int out_dtype, int sms,
                                  cudaStream_t stream) {
  if (dtype == RD_F32)
    return out_dtype == RD_F32 ? fwd_by_width<float, float>(a, sms, stream)
                               : fwd_by_width<float, bf16>(a, sms, stream);
  return out_dtype == RD_F32 ? fwd_by_width<bf16, float>(a, sms, stream)
                             : fwd_by_width<bf16, bf16>(a, sms, stream);
}

// us in one launch / in two, bf16: 256 x 256 2.5 / 4.6, 512 x 1024 3.2 / 7.2, 512 x 4096 5.7 / 10.4, 1024 x 4096 12.1 / 12.6, 1024 x 8192
// 15.6 / 16.4, but 2048 x 256 9.8 / 7.7, 2048 x 4096 22.8 / 16.7
bool layer_norm_bwd_few(int64_t rows, int64_t hidden) { return rows <= 1024 && hidden <= 8192; }

// the most that the kernels write: as many clusters as fit the SMs' threads, and no more than the rows fill
int layer_norm_bwd_parts(int64_t rows, int64_t hidden, int sms) {
  if (layer_norm_bwd_few(rows, hidden)) return 0;
  const BwdShape shape = bwd_shape(hidden);
  int64_t p, most;
  if (shape.rows == 0) {
    p = ceil_of(rows, 64);
    most = 64;
  } else {
    const int cluster = shape.split > 1 ? shape.split : kNormCluster;
    p = ceil_of(rows, shape.split > 1 ? shape.rows : kNormCluster * shape.rows);
    most = ceil_of(static_cast<int64_t>(sms) * shape.blocks, cluster);
  }
  return static_cast<int>(p < 1 ? 1 : (p < most ? p : most));
}

cudaError_t launch_layer_norm_bwd(const NormArgs& a, int dtype, int out_dtype, int sms,
                                  cudaStream_t stream) {
  int parts = layer_norm_bwd_parts(a.rows, a.hidden, sms);
  cudaError_t e;
  if (dtype == RD_F32)
    e = out_dtype == RD_F32 ? bwd_by_width<float, float>(a, &parts, sms, stream)
                            : bwd_by_width<float, bf16>(a, &parts, sms, stream);
  else
    e = out_dtype == RD_F32 ? bwd_by_width<bf16, float>(a, &parts, sms, stream)
                            : bwd_by_width<bf16, bf16>(a, &parts, sms, stream);
  if (e != cudaSuccess || a.parts == nullptr || parts == 0) return e;
  return launch_pdl(layer_norm_parts_kernel, dim3(static_cast<unsigned>(ceil_of(2 * static_cast<int64_t>(a.hidden), 32))),
                    32 * kPartLanes, 0, 1, stream, a, static_cast<int32_t>(parts));
}

}  // namespace rd
