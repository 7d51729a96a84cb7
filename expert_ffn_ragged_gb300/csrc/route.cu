// route.cu -- the router: scores, expert choice and weights of each token, and the gradient of
// the logits from the gradient of the weights.
//
// One warp owns a token; lane l holds the EPL consecutive experts from l * EPL in registers, so a
// row is read in 16-byte vectors and a lower lane always means a lower expert index.
//
// Choice: the lanes put their largest keys in shared memory and count which of them are larger; no key
// below the topk-th largest of these can be chosen, and the few that are left (hardly more than
// topk) are gathered and ranked against each other by counting again.  Popping the best key topk
// times, with the keys of a lane sorted first, took 1.6 times the instructions.  The two largest keys
// of a group that is a power of two of whole lanes are merged by exchanges among these.
//
// Bound: instructions, not memory: 32771 tokens, 256 experts in 8 groups, sigmoid, top-8, f32 logits
// (36.7 MB: 5.4 us at the measured copy rate) take 26.2 us, with the issue slots 68 % busy and DRAM 14 %;
// the exp and the reciprocal of the sigmoid, whose exact f32 values the choice is defined by, are a
// third of the instructions.  The gradient, 65536 x 128 softmax over all: 71.3 MB in 16.7 to 17.4 us
// (4.2 TB/s; issue 65 %).  One token with its plan: 6.2 us, two dependent launches.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "launch.h"
#include "moe_args.h"
#include "route_math.cuh"

namespace rd {
namespace {

constexpr int kRouteWarps = 8;
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kLow = -INFINITY;  // key of a masked expert

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ int32_t tokens_below(const int32_t* limit, int32_t tokens) {
  if (limit == nullptr) return tokens;
  const int32_t v = *limit;
  return v < 0 ? 0 : (v > tokens ? tokens : v);
}

// the logistic in the elementwise f32 arithmetic that the keys are defined by
__device__ __forceinline__ float sigmoid_f32(float l) { return __frcp_rn(__fadd_rn(1.0f, expf(-l))); }

// The same for a lane's logits, NaN for a masked one (d is infinite, and infinity times 0 is NaN in the
// step), with one test for those so negative that 1 / d leaves the normal numbers (a test for each made
// the branches as expensive as the arithmetic).
template <int EPL>
__device__ __forceinline__ void sigmoids_f32(const float (&l)[EPL], float (&s)[EPL]) {
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const float d = __fadd_rn(1.0f, expf(-l[i]));
    s[i] = reciprocal_fast(d);
    most = fmaxf(most, l[i] > kLow ? d : 0.0f);  // -inf is masked, whatever its sigmoid
  }
  if (!(most < kFastRcp)) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = l[i] > kLow ? sigmoid_f32(l[i]) : NAN;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// maximum over the warp; NaN operands lose
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ bool is_masked(float l) { return !(l > kLow); }

// This lane's EPL logits of a row; experts past the end read as -inf.  `vec`: rows and lanes start
// on boundaries of the vectors used here.
template <int EPL>
__device__ __forceinline__ void load_row(const float* row, int e0, int experts, bool vec, float (&v)[EPL]) {
  if (EPL % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      float4 x = make_float4(kLow, kLow, kLow, kLow);
      if (e0 + i < experts) x = *reinterpret_cast<const float4*>(row + e0 + i);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = e0 + i < experts ? row[e0 + i] : kLow;
  }
}

template <int EPL>
__device__ __forceinline__ void load_row(const __nv_bfloat16* row, int e0, int experts, bool vec,
                                         float (&v)[EPL]) {
  if (EPL % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      uint2 x = make_uint2(0xFF80FF80u, 0xFF80FF80u);
      if (e0 + i < experts) x = *reinterpret_cast<const uint2*>(row + e0 + i);
      v[i] = __uint_as_float(x.x << 16);
      v[i + 1] = __uint_as_float(x.x & 0xFFFF0000u);
      v[i + 2] = __uint_as_float(x.y << 16);
      v[i + 3] = __uint_as_float(x.y & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = e0 + i < experts ? load_logit(row + e0 + i) : kLow;
  }
}

template <int EPL>
__device__ __forceinline__ void store_row(float* row, int e0, int experts, bool vec, const float (&v)[EPL]) {
  if (EPL % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4)
      if (e0 + i < experts)
        *reinterpret_cast<float4*>(row + e0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e0 + i < experts) row[e0 + i] = v[i];
  }
}

template <int EPL>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int e0, int experts, bool vec,
                                          const float (&v)[EPL]) {
  if (EPL % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v[i], v[i + 1]);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(v[i + 2], v[i + 3]);
      if (e0 + i < experts)
        *reinterpret_cast<uint2*>(row + e0 + i) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                             *reinterpret_cast<const uint32_t*>(&hi));
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e0 + i < experts) row[e0 + i] = __float2bfloat16_rn(v[i]);
  }
}

// What a slot's weight is made of, in the lane that holds the slot: part (its exp or sigmoid) and
// the warp-wide sum it is divided by (1 for sigmoid scores as they are).  ex: the exps of this
// lane's logits, filled for softmax scores over all experts.
template <int EPL, int SCORE>
__device__ __forceinline__ void slot_parts(const RouteArgs& a, bool there, float at,
                                           const float (&logit)[EPL], float (&ex)[EPL], float& part,
                                           float& total) {
  if (SCORE == RD_SCORE_SOFTMAX) {
    float top = there ? at : kLow;
    if (!a.renormalize) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) top = fmaxf(top, logit[i]);  // a NaN logit loses
    }
      top = warp_max(top);
    part = there ? expf(at - top) : 0.0f;
    float sum = part;
    if (!a.renormalize) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        ex[i] = is_masked(logit[i]) ? 0.0f : expf(logit[i] - top);
        sum += ex[i];
      }
    }
    total = warp_sum(sum);
  } else {
    part = there ? sigmoid_f32(at) : 0.0f;
    total = a.renormalize ? warp_sum(part) : 1.0f;
  }
}

// Shared memory (words): the biases, then per warp the keys of the candidates (and four that never
// win), their experts, the chosen ids, and the values that are ranked by counting.
constexpr int route_warp_words(int epl) { return 32 * epl + 4 + 32 * epl + 4 + 32 + 32; }
constexpr size_t route_smem_bytes(int epl) {
  return sizeof(float) * (32 * epl + kRouteWarps * route_warp_words(epl));
}

// How many of the n values (a multiple of four, in shared memory) are larger than v; none of them is -0.
__device__ __forceinline__ int count_larger(const float* values, int n, float v) {
  int c = 0;
#pragma unroll 8
  for (int j = 0; j < n; j += 4) {
    const float4 o = *reinterpret_cast<const float4*>(values + j);
    // the sign of a difference (never rounded to zero) in place of a comparison and a select
    c += static_cast<int>(__float_as_uint(v - o.x) >> 31) + static_cast<int>(__float_as_uint(v - o.y) >> 31) +
         static_cast<int>(__float_as_uint(v - o.z) >> 31) + static_cast<int>(__float_as_uint(v - o.w) >> 31);
  }
  return c;
}

// EPL values of shared memory, from a boundary of EPL
template <int EPL>
__device__ __forceinline__ void load_shared(const float* p, float (&v)[EPL]) {
  if (EPL % 4 == 0) {
#pragma unroll
    for (int i = 0; i + 3 < EPL; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = p[i];
  }
}

template <int EPL, class T, int SCORE>
__global__ void __launch_bounds__(kRouteWarps * 32, EPL <= 8 ? 4 : 1) route_kernel(const RouteArgs a) {
  extern __shared__ __align__(16) float smem_route[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* sbias = smem_route;
  float* ckey = sbias + 32 * EPL + warp * route_warp_words(EPL);
  int* cexp = reinterpret_cast<int*>(ckey + 32 * EPL + 4);
  int* chosen = cexp + 32 * EPL + 4;
  float* ranked = reinterpret_cast<float*>(chosen + 32);
  pdl_trigger();
  pdl_wait();
  if (a.bias != nullptr) {
    for (int e = threadIdx.x; e < 32 * EPL; e += kRouteWarps * 32) sbias[e] = e < a.experts ? a.bias[e] : 0.0f;
    __syncthreads();
  }
  const int32_t L = tokens_below(a.limit, a.tokens);
  const T* logits = static_cast<const T*>(a.logits);
  const int gsize = a.experts / a.groups;
  const int e0 = lane * EPL;
  // the lanes of a group, where groups are a power of two of whole lanes
  const int lpg = gsize / EPL;
  const bool lane_groups = gsize % EPL == 0 && (lpg & (lpg - 1)) == 0;
  const int my_group = lane_groups ? lane / lpg : 0;
  // Near 2^31 tokens t + stride leaves 32 bits: `last` decides whether there is a next token, and the step
  // after the last one is unsigned.
  const int stride = gridDim.x * kRouteWarps, last = L - stride;
  int t = blockIdx.x * kRouteWarps + warp;
  float next[EPL];
  if (t < L) load_row<EPL>(logits + static_cast<int64_t>(t) * a.experts, e0, a.experts, a.vec, next);
  for (bool more = t < L; more; t += static_cast<uint32_t>(stride)) {
    const T* row = logits + static_cast<int64_t>(t) * a.experts;
    float logit[EPL], key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) logit[i] = next[i];
    more = t < last;
    if (more)  // the next token's row, under this one's work
      load_row<EPL>(row + static_cast<int64_t>(stride) * a.experts, e0, a.experts, a.vec, next);
    if (SCORE == RD_SCORE_SIGMOID) {
      sigmoids_f32<EPL>(logit, key);
    } else {
      // -0 + 0 is 0: the ranking below takes the sign of a difference, which tells zeros of unlike signs
      // apart.  A sum with a bias is no -0 then either, and a sigmoid never is.
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = __fadd_rn(logit[i], 0.0f);
    }
    if (a.bias != nullptr) {
      float b[EPL];
      load_shared<EPL>(sbias + e0, b);
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = __fadd_rn(key[i], b[i]);
    }
    // a masked expert's key is -inf or NaN by itself
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = fmaxf(key[i], kLow);
    float mine1 = key[0];  // this lane's largest key
    if (a.groups > 1 && lane_groups) {
      float mine2 = kLow;
#pragma unroll
      for (int i = 1; i < EPL; ++i) {
        mine2 = fmaxf(mine2, fminf(mine1, key[i]));
        mine1 = fmaxf(mine1, key[i]);
      }
      // the group's two largest keys, merged among its lanes
      float first = mine1, second = mine2;
      for (int d = 1; d < lpg; d <<= 1) {
        const float f = __shfl_xor_sync(kAll, first, d), g = __shfl_xor_sync(kAll, second, d);
        second = fmaxf(fmaxf(second, g), fminf(first, f));
        first = fmaxf(first, f);
      }
      float score = first;
      if (SCORE == RD_SCORE_SIGMOID && second > kLow) score = __fadd_rn(first, second);
      // the groups before this one: those with a larger score, and of equal ones the lower
      ranked[lane] = kLow;
      __syncwarp();
      if (lane % lpg == 0 && my_group < a.groups) ranked[my_group] = score;
      __syncwarp();
      int before = 0;
      for (int g = 0; g < a.groups; g += 4) {
        const float4 o = *reinterpret_cast<const float4*>(ranked + g);
        before += (o.x > score || (o.x == score && g < my_group)) +
                  (o.y > score || (o.y == score && g + 1 < my_group)) +
                  (o.z > score || (o.z == score && g + 2 < my_group)) +
                  (o.w > score || (o.w == score && g + 3 < my_group));
      }
      __syncwarp();
      const bool kept = before < a.topk_groups;  // one without an expert has no key to offer
      if (!kept) {
        mine1 = kLow;
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = kLow;
      }
    } else {
      if (a.groups > 1) {
        // groups across lane boundaries: lane g scores group g from shared memory
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (e0 + i < a.experts) ckey[e0 + i] = key[i];
        __syncwarp();
        float score = kLow;
        if (lane < a.groups) {
          float first = kLow, second = kLow;
          for (int e = lane * gsize; e < (lane + 1) * gsize; ++e) {
            const float v = ckey[e];
            second = fmaxf(second, fminf(first, v));
            first = fmaxf(first, v);
          }
          score = first;
          if (SCORE == RD_SCORE_SIGMOID && second > kLow) score = __fadd_rn(first, second);
        }
        uint32_t kept = 0;
        for (int r = 0; r < a.topk_groups; ++r) {
          const float best = warp_max(score);
          if (!(best > kLow)) break;
          const int g = __ffs(__ballot_sync(kAll, score == best)) - 1;
          kept |= 1u << g;
          if (lane == g) score = kLow;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (e0 + i < a.experts && !((kept >> ((e0 + i) / gsize)) & 1u)) key[i] = kLow;
        mine1 = key[0];
      }
#pragma unroll
      for (int i = 1; i < EPL; ++i) mine1 = fmaxf(mine1, key[i]);
    }
    // tau: the topk-th largest of the lanes' largest keys.  Where fewer lanes have one, every key
    // that is not -inf is a candidate.
    ranked[lane] = mine1;
    __syncwarp();
    const bool among = count_larger(ranked, 32, mine1) < a.topk;
    const float tau = fmaxf(-warp_max(among ? -mine1 : kLow), -3.402823466e38f);
    // the candidates, in the order of their experts
    int count = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) count += key[i] >= tau ? 1 : 0;
    int at = count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kAll, at, d);
      if (lane >= d) at += o;
    }
    const int total_c = __shfl_sync(kAll, at, 31);
    at -= count;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool in = key[i] >= tau;
      if (in) ckey[at] = key[i];
      if (in) cexp[at] = e0 + i;
      at += in ? 1 : 0;
    }
    if (lane < 4) ckey[total_c + lane] = kLow;
    chosen[lane] = -1;
    __syncwarp();
    // a candidate's rank: those with a larger key; equal ones, which then meet at one rank, are told
    // apart by their order
    const int padded = (total_c + 3) & ~3;
    if (total_c <= 32) {
      const float mine = lane < total_c ? ckey[lane] : kLow;
      int rank = count_larger(ckey, padded, mine);
      const unsigned mine_at = lane < total_c ? 1u << rank : 0u;
      if (__popc(__reduce_or_sync(kAll, mine_at)) != total_c) {
        for (int j = 0; j < total_c; ++j) rank += j < lane && ckey[j] == mine ? 1 : 0;
      }
      if (lane < total_c && rank < a.topk) chosen[rank] = cexp[lane];
    } else {
      for (int c = lane; c < total_c; c += 32) {
        const float mine = ckey[c];
        int rank = count_larger(ckey, padded, mine);
        for (int j = 0; j < c; ++j) rank += ckey[j] == mine ? 1 : 0;
        if (rank < a.topk) chosen[rank] = cexp[c];
      }
    }
    __syncwarp();
    const int my_id = lane < a.topk ? chosen[lane] : -1;
    const bool there = my_id >= 0;
    const float own = there ? load_logit(row + my_id) : 0.0f;
    float part, total, ex[EPL];
    slot_parts<EPL, SCORE>(a, there, own, logit, ex, part, total);
    if (lane < a.topk) {
      const int64_t o = static_cast<int64_t>(t) * a.topk + lane;
      a.ids[o] = my_id;
      // !(total <= 0) lets a NaN sum through
      a.weights[o] = there && !(total <= 0.0f) ? __fmul_rn(__fdiv_rn(part, total), a.scale) : 0.0f;
    }
    __syncwarp();  // the candidates are read: the next token may write its own
  }
}

// The row's gradients are put together in shared memory, where the chosen experts add theirs to
// what every expert gets, and leave in vectors.
template <int EPL, class T, int SCORE>
__global__ void __launch_bounds__(kRouteWarps * 32) route_bwd_kernel(const RouteArgs a) {
  extern __shared__ __align__(16) float smem_rows[];  // [warps][32 * EPL]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* srow = smem_rows + warp * 32 * EPL;
  pdl_trigger();
  pdl_wait();
  const int32_t L = tokens_below(a.limit, a.tokens);
  const bool dense = SCORE == RD_SCORE_SOFTMAX && !a.renormalize;
  const int e0 = lane * EPL;
  const int stride = gridDim.x * kRouteWarps, last = L - stride;  // as above
  const T* logits = static_cast<const T*>(a.logits);
  int t = blockIdx.x * kRouteWarps + warp;
  float next[EPL];
  int next_id = -1;
  float next_d = 0.0f;
  auto fetch = [&](int tt) {
    if (dense) load_row<EPL>(logits + static_cast<int64_t>(tt) * a.experts, e0, a.experts, a.vec, next);
    if (lane < a.topk) {
      const int64_t o = static_cast<int64_t>(tt) * a.topk + lane;
      next_id = a.ids[o];
      next_d = a.d_weights[o];
    }
  };
  if (t < L) fetch(t);
  for (bool more = t < L; more; t += static_cast<uint32_t>(stride)) {
    const T* row = logits + static_cast<int64_t>(t) * a.experts;
    T* out = static_cast<T*>(a.d_logits) + static_cast<int64_t>(t) * a.experts;
    float logit[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) logit[i] = dense ? next[i] : kLow;
    const int id = next_id;
    const bool there = lane < a.topk && id >= 0 && id < a.experts;
    const float d = there ? next_d : 0.0f;
    const float at = there ? load_logit(row + id) : 0.0f;
    more = t < last;
    if (more) fetch(t + stride);
    float part, total, ex[EPL];
    slot_parts<EPL, SCORE>(a, there, at, logit, ex, part, total);
    // A softmax sum is 1 .. experts (0 without an expert, NaN with a +inf logit).  One of sigmoids may be a
    // subnormal number: its reciprocal, and d / sum, would be infinite where the share and the gradient are not.
    const float inv = SCORE == RD_SCORE_SOFTMAX && !(total <= 0.0f) ? reciprocal_fast(total) : 0.0f;
    // a quotient, so that a slot that is all of the sum has weight one and a gradient of exactly zero
    const float q = SCORE == RD_SCORE_SOFTMAX ? part * inv : (total <= 0.0f ? 0.0f : __fdiv_rn(part, total));
    const float mean = warp_sum(there ? q * d : 0.0f);
    float v[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      // 0 * NaN: a masked expert's gradient is 0 whatever the others are
      v[i] = dense && !is_masked(logit[i]) ? -a.scale * (ex[i] * inv) * mean : 0.0f;
      if (EPL % 4 != 0) srow[e0 + i] = v[i];
    }
    if (EPL % 4 == 0) {
#pragma unroll
      for (int i = 0; i + 3 < EPL; i += 4)
        *reinterpret_cast<float4*>(srow + e0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
    __syncwarp();
    if (there) {
      float g;
      if (SCORE == RD_SCORE_SOFTMAX) g = a.scale * q * (d - mean);
      else g = a.scale * (a.renormalize ? q * (d - mean) : d * part) * (1.0f - part);
      srow[id] = g;
    }
    __syncwarp();
    if (EPL % 4 == 0) {
#pragma unroll
      for (int i = 0; i + 3 < EPL; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(srow + e0 + i);
        v[i] = x.x;
        v[i + 1] = x.y;
        v[i + 2] = x.z;
        v[i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = srow[e0 + i];
    }
    store_row<EPL>(out, e0, a.experts, a.vec, v);
    __syncwarp();
  }
}

template <int EPL, class T, int SCORE>
cudaError_t launch_score(RouteArgs a, bool bwd, int sms, cudaStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(a.tokens) + kRouteWarps - 1) / kRouteWarps;
  // blocks an SM: two rounds of the four that fit (route), two of the six that fit (its gradient; with
  // 8 the second round is a third full: 65536 x 128 17.7 us against 16.9)
  const int most = sms * (bwd ? 12 : 8);
  const int grid = static_cast<int>(blocks < most ? blocks : most);
  // rows and lanes start on vector boundaries (16 bytes of f32, 8 of bf16: four elements)
  const uintptr_t unit = 4 * sizeof(T);
  a.vec = a.experts % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % unit == 0 &&
          reinterpret_cast<uintptr_t>(a.d_logits) % unit == 0;
  if (bwd) {
    return launch_pdl(route_bwd_kernel<EPL, T, SCORE>, dim3(grid), kRouteWarps * 32,
                      sizeof(float) * kRouteWarps * 32 * EPL, 1, stream, a);
  }
  constexpr size_t smem = route_smem_bytes(EPL);
  if (smem > 48 * 1024) {
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev].load(std::memory_order_acquire)) {
      const cudaError_t e = cudaFuncSetAttribute(
          route_kernel<EPL, T, SCORE>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return e;
      attr_set[dev].store(true, std::memory_order_release);
    }
  }
  return launch_pdl(route_kernel<EPL, T, SCORE>, dim3(grid), kRouteWarps * 32, smem, 1, stream, a);
}

template <int EPL, class T>
cudaError_t launch_epl(const RouteArgs& a, bool bwd, int sms, cudaStream_t stream) {
  return a.score == RD_SCORE_SOFTMAX ? launch_score<EPL, T, RD_SCORE_SOFTMAX>(a, bwd, sms, stream)
                                     : launch_score<EPL, T, RD_SCORE_SIGMOID>(a, bwd, sms, stream);
}

template <class T>
cudaError_t launch_t(const RouteArgs& a, bool bwd, int sms, cudaStream_t stream) {
  const int epl = (a.experts + 31) / 32;
  if (epl <= 1) return launch_epl<1, T>(a, bwd, sms, stream);
  if (epl <= 2) return launch_epl<2, T>(a, bwd, sms, stream);
  if (epl <= 4) return launch_epl<4, T>(a, bwd, sms, stream);
  if (epl <= 8) return launch_epl<8, T>(a, bwd, sms, stream);
  if (epl <= 16) return launch_epl<16, T>(a, bwd, sms, stream);
  return launch_epl<32, T>(a, bwd, sms, stream);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, int dtype, int sms, cudaStream_t stream) {
  return dtype == RD_F32 ? launch_t<float>(a, false, sms, stream)
                         : launch_t<__nv_bfloat16>(a, false, sms, stream);
}

cudaError_t launch_route_bwd(const RouteArgs& a, int dtype, int sms, cudaStream_t stream) {
  return dtype == RD_F32 ? launch_t<float>(a, true, sms, stream)
                         : launch_t<__nv_bfloat16>(a, true, sms, stream);
}

}  // namespace rd
