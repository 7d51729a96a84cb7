// route.cu -- the router: scores, expert choice and weights of each token, and the gradient of
// the logits from the gradient of the weights.
//
// One warp owns a token; lane l holds the EPL consecutive experts from l * EPL in registers, so a
// row is read in 16-byte vectors and a lower lane always means a lower expert index.
//
// Choice: up to 8 keys a lane are sorted once (a network of stable compare-exchanges), and each of
// the topk rounds is one warp-wide maximum of the lanes' heads, a ballot for the lowest lane that
// has it, and a pop in that lane.  More keys a lane (over 256 experts) are scanned in every round,
// as sorting them would cost more than the rounds.  The two largest keys of a group, where groups are whole lanes, are two
// maxima over the group's lanes.
//
// Bound: instructions, not memory.  At 32771 x 256 in f32 (36.7 MB: 5.4 us at the measured copy
// rate) a token costs some 500 warp instructions, a third of them the exp and the reciprocal of
// the sigmoid, whose exact f32 values the choice is defined by.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_args.h"

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

// the logistic in the elementwise f32 arithmetic that the keys are defined by (a correctly rounded
// reciprocal is the division 1 / x)
__device__ __forceinline__ float sigmoid_f32(float l) { return __frcp_rn(__fadd_rn(1.0f, expf(-l))); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// maximum over the lanes of `mask` (which names the calling lane); NaN operands lose
__device__ __forceinline__ float lanes_max(float v, unsigned mask) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "r"(mask));
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
      if (e0 + i < experts) x = __ldg(reinterpret_cast<const float4*>(row + e0 + i));
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = e0 + i < experts ? __ldg(row + e0 + i) : kLow;
  }
}

template <int EPL>
__device__ __forceinline__ void load_row(const __nv_bfloat16* row, int e0, int experts, bool vec,
                                         float (&v)[EPL]) {
  if (EPL % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      uint2 x = make_uint2(0xFF80FF80u, 0xFF80FF80u);
      if (e0 + i < experts) x = __ldg(reinterpret_cast<const uint2*>(row + e0 + i));
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

constexpr int kSortedKeys = 8;  // keys a lane sorts rather than scans

// Sort this lane's keys, largest first, equal keys by index: an odd-even transposition network
// (only neighbours are exchanged, and only when strictly out of order, which keeps it stable).
template <int EPL>
__device__ __forceinline__ void sort_keys(float (&key)[EPL], int (&idx)[EPL]) {
#pragma unroll
  for (int round = 0; round < EPL; ++round) {
#pragma unroll
    for (int i = round & 1; i + 1 < EPL; i += 2) {
      const bool swap = key[i] < key[i + 1];
      const float a = swap ? key[i + 1] : key[i], b = swap ? key[i] : key[i + 1];
      const int ia = swap ? idx[i + 1] : idx[i], ib = swap ? idx[i] : idx[i + 1];
      key[i] = a;
      key[i + 1] = b;
      idx[i] = ia;
      idx[i + 1] = ib;
    }
  }
}

// What a slot's weight is made of, in the lane that holds the slot: part (its exp or sigmoid) and
// the warp-wide sum it is divided by (1 for sigmoid scores as they are).  ex: the exps of this
// lane's logits, filled for softmax scores over all experts.
template <int EPL>
__device__ __forceinline__ void slot_parts(const RouteArgs& a, bool there, float at,
                                           const float (&logit)[EPL], float (&ex)[EPL], float& part,
                                           float& total) {
  if (a.score == RD_SCORE_SOFTMAX) {
    float top = there ? at : kLow;
    if (!a.renormalize) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) top = fmaxf(top, logit[i]);  // a NaN logit loses
    }
    top = lanes_max(top, kAll);
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

template <int EPL, class T>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteArgs a) {
  extern __shared__ float smem_keys[];  // [warps][experts], for groups that are not whole lanes
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t L = tokens_below(a.limit, a.tokens);
  const T* logits = static_cast<const T*>(a.logits);
  const int gsize = a.experts / a.groups;
  const int e0 = lane * EPL;
  const bool lane_groups = gsize % EPL == 0;
  // the lanes of this lane's group
  const int lpg = lane_groups ? gsize / EPL : 1;
  const int my_group = lane / lpg;
  const unsigned group_mask = (lpg >= 32 ? kAll : ((1u << lpg) - 1u)) << (my_group * lpg);
  float bias[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    bias[i] = a.bias != nullptr && e0 + i < a.experts ? a.bias[e0 + i] : 0.0f;
  const int stride = gridDim.x * kRouteWarps;
  int t = blockIdx.x * kRouteWarps + warp;
  float next[EPL];
  if (t < L) load_row<EPL>(logits + static_cast<int64_t>(t) * a.experts, e0, a.experts, a.vec, next);
  for (; t < L; t += stride) {
    const T* row = logits + static_cast<int64_t>(t) * a.experts;
    float logit[EPL], key[EPL];
    int idx[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) logit[i] = next[i];
    if (t + stride < L)  // the next token's row, under this one's work
      load_row<EPL>(row + static_cast<int64_t>(stride) * a.experts, e0, a.experts, a.vec, next);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      float k = a.score == RD_SCORE_SOFTMAX ? logit[i] : sigmoid_f32(logit[i]);
      if (a.bias != nullptr) k = __fadd_rn(k, bias[i]);
      key[i] = is_masked(logit[i]) || is_masked(k) ? kLow : k;
      idx[i] = i;
    }
    if (a.groups > 1 && !lane_groups) {
      // groups across lane boundaries: lane g scores group g from shared memory, and the experts
      // of the groups that are not kept are masked before the sort
      float* sk = smem_keys + warp * a.experts;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (e0 + i < a.experts) sk[e0 + i] = key[i];
      __syncwarp();
      float score = kLow;
      if (lane < a.groups) {
        float first = kLow, second = kLow;
        for (int e = lane * gsize; e < (lane + 1) * gsize; ++e) {
          const float v = sk[e];
          second = fmaxf(second, fminf(first, v));
          first = fmaxf(first, v);
        }
        score = first;
        if (a.score == RD_SCORE_SIGMOID && second > kLow) score = __fadd_rn(first, second);
      }
      uint32_t kept = 0;
      for (int r = 0; r < a.topk_groups; ++r) {
        const float best = lanes_max(score, kAll);
        if (!(best > kLow)) break;
        const int g = __ffs(__ballot_sync(kAll, score == best)) - 1;
        kept |= 1u << g;
        if (lane == g) score = kLow;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (e0 + i < a.experts && !((kept >> ((e0 + i) / gsize)) & 1u)) key[i] = kLow;
    }
    constexpr bool kSorted = EPL <= kSortedKeys;
    if (kSorted) sort_keys<EPL>(key, idx);
    if (a.groups > 1 && lane_groups) {
      // the group's largest key; then its second largest, for which the (lowest) lane that has
      // the largest offers its own second
      float score = kLow;
      if (my_group < a.groups) {
        float mine1 = key[0], mine2 = kLow;
        if (kSorted) {
          if (EPL > 1) mine2 = key[EPL > 1 ? 1 : 0];
        } else {
#pragma unroll
          for (int i = 1; i < EPL; ++i) {
            mine2 = fmaxf(mine2, fminf(mine1, key[i]));
            mine1 = fmaxf(mine1, key[i]);
          }
        }
        const float first = lanes_max(mine1, group_mask);
        score = first;
        if (a.score == RD_SCORE_SIGMOID) {
          const unsigned has = __ballot_sync(group_mask, mine1 == first);
          const float offer = lane == __ffs(has & group_mask) - 1 ? mine2 : mine1;
          const float second = lanes_max(offer, group_mask);
          if (second > kLow) score = __fadd_rn(first, second);
        }
      }
      __syncwarp();
      bool mine = false;
      for (int r = 0; r < a.topk_groups; ++r) {
        const float best = lanes_max(score, kAll);
        if (!(best > kLow)) break;
        const int g = (__ffs(__ballot_sync(kAll, score == best)) - 1) / lpg;
        if (my_group == g) {
          mine = true;
          score = kLow;
        }
      }
      if (!mine) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = kLow;
      }
    }
    int my_id = -1;
    for (int k = 0; k < a.topk; ++k) {
      float head = key[0];
      if (!kSorted) {
#pragma unroll
        for (int i = 1; i < EPL; ++i) head = fmaxf(head, key[i]);
      }
      const float best = lanes_max(head, kAll);
      if (!(best > kLow)) break;
      const int owner = __ffs(__ballot_sync(kAll, head == best)) - 1;
      int at = idx[0];
      if (kSorted) {
        if (lane == owner) {
#pragma unroll
          for (int i = 0; i + 1 < EPL; ++i) {
            key[i] = key[i + 1];
            idx[i] = idx[i + 1];
          }
          key[EPL - 1] = kLow;
        }
      } else {
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i)
          if (key[i] == best) at = i;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (lane == owner && i == at) key[i] = kLow;
      }
      const int e = owner * EPL + __shfl_sync(kAll, at, owner);
      if (lane == k) my_id = e;
    }
    const bool there = my_id >= 0;
    const float at = there ? load_logit(row + my_id) : 0.0f;
    float part, total, ex[EPL];
    slot_parts<EPL>(a, there, at, logit, ex, part, total);
    if (lane < a.topk) {
      const int64_t o = static_cast<int64_t>(t) * a.topk + lane;
      a.ids[o] = my_id;
      // !(total <= 0) lets a NaN sum through
      a.weights[o] = there && !(total <= 0.0f) ? __fmul_rn(__fdiv_rn(part, total), a.scale) : 0.0f;
    }
  }
}

// The row's gradients are put together in shared memory, where the chosen experts add theirs to
// what every expert gets, and leave in vectors.
template <int EPL, class T>
__global__ void __launch_bounds__(kRouteWarps * 32) route_bwd_kernel(const RouteArgs a) {
  extern __shared__ __align__(16) float smem_rows[];  // [warps][32 * EPL]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* srow = smem_rows + warp * 32 * EPL;
  const int32_t L = tokens_below(a.limit, a.tokens);
  const bool dense = a.score == RD_SCORE_SOFTMAX && !a.renormalize;
  const int e0 = lane * EPL;
  const int stride = gridDim.x * kRouteWarps;
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
  for (; t < L; t += stride) {
    const T* row = logits + static_cast<int64_t>(t) * a.experts;
    T* out = static_cast<T*>(a.d_logits) + static_cast<int64_t>(t) * a.experts;
    float logit[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) logit[i] = dense ? next[i] : kLow;
    const int id = next_id;
    const bool there = lane < a.topk && id >= 0 && id < a.experts;
    const float d = there ? next_d : 0.0f;
    const float at = there ? load_logit(row + id) : 0.0f;
    if (t + stride < L) fetch(t + stride);
    float part, total, ex[EPL];
    slot_parts<EPL>(a, there, at, logit, ex, part, total);
    const float inv = !(total <= 0.0f) ? __fdiv_rn(1.0f, total) : 0.0f;
    const float q = part * inv;
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
      if (a.score == RD_SCORE_SOFTMAX) g = a.scale * q * (d - mean);
      else g = a.scale * (a.renormalize ? (d - mean) * inv : d) * part * (1.0f - part);
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

template <int EPL, class T>
cudaError_t launch_epl(RouteArgs a, bool bwd, int sms, cudaStream_t stream) {
  const int64_t blocks = (a.tokens + kRouteWarps - 1) / kRouteWarps;
  const int grid = static_cast<int>(blocks < sms * 8 ? blocks : sms * 8);
  // rows and lanes start on vector boundaries (16 bytes of f32, 8 of bf16: four elements)
  const uintptr_t unit = 4 * sizeof(T);
  a.vec = a.experts % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % unit == 0 &&
          reinterpret_cast<uintptr_t>(a.d_logits) % unit == 0;
  if (bwd) {
    route_bwd_kernel<EPL, T><<<grid, kRouteWarps * 32, sizeof(float) * kRouteWarps * 32 * EPL, stream>>>(a);
  } else {
    const bool shared = a.groups > 1 && (a.experts / a.groups) % EPL != 0;
    route_kernel<EPL, T><<<grid, kRouteWarps * 32, shared ? sizeof(float) * kRouteWarps * a.experts : 0,
                           stream>>>(a);
  }
  return cudaGetLastError();
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
