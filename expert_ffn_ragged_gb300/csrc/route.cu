// route.cu -- the router: scores, expert choice and weights of each token, and the gradient of
// the logits from the gradient of the weights.
//
// One warp owns a token; its logits sit in registers, expert e in lane e % 32.  The choice works
// on order-preserving integer keys (a float's bits with the sign folded in), so that each of the
// topk rounds is two warp reductions: the largest key, then the lowest index that has it.
// Memory: the logits once (T * E elements), 8 bytes a slot.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_args.h"

namespace rd {
namespace {

constexpr int kRouteWarps = 8;
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ int32_t tokens_below(const int32_t* limit, int32_t tokens) {
  if (limit == nullptr) return tokens;
  const int32_t v = *limit;
  return v < 0 ? 0 : (v > tokens ? tokens : v);
}

// the logistic in the elementwise f32 arithmetic that the keys are defined by
__device__ __forceinline__ float sigmoid_f32(float l) {
  return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l)));
}

// order-preserving integer of a key; 0 for a masked expert (and for a key of -inf or NaN)
__device__ __forceinline__ uint32_t order_key(float key, bool masked) {
  if (masked || !(key > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(key + 0.0f);  // -0 and +0 tie
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_of_order(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}

__device__ __forceinline__ bool is_masked(float l) { return !(l > -INFINITY); }

// What a slot's weight is made of, in the lane that holds the slot: part (its exp or sigmoid) and
// the warp-wide sum it is divided by (1 for sigmoid scores as they are).
template <int EPL>
__device__ __forceinline__ void slot_parts(const RouteArgs& a, bool there, float at,
                                           const float (&logit)[EPL], float& part, float& total) {
  if (a.score == RD_SCORE_SOFTMAX) {
    float top = there ? at : -INFINITY;
    if (!a.renormalize) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (!is_masked(logit[i])) top = fmaxf(top, logit[i]);
    }
    top = warp_max(top);
    part = there ? expf(at - top) : 0.0f;
    float sum = part;
    if (!a.renormalize) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (!is_masked(logit[i])) sum += expf(logit[i] - top);
    }
    total = warp_sum(sum);
  } else {
    part = there ? sigmoid_f32(at) : 0.0f;
    total = a.renormalize ? warp_sum(part) : 1.0f;
  }
}

template <int EPL, class T>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteArgs a) {
  extern __shared__ uint32_t smem_keys[];  // [warps][experts], with expert groups only
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t L = tokens_below(a.limit, a.tokens);
  const T* logits = static_cast<const T*>(a.logits);
  const int gsize = a.experts / a.groups;
  for (int t = blockIdx.x * kRouteWarps + warp; t < L; t += gridDim.x * kRouteWarps) {
    const T* row = logits + static_cast<int64_t>(t) * a.experts;
    float logit[EPL];
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      logit[i] = e < a.experts ? load_logit(row + e) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      float k = a.score == RD_SCORE_SOFTMAX ? logit[i] : sigmoid_f32(logit[i]);
      if (a.bias != nullptr && e < a.experts) k = __fadd_rn(k, a.bias[e]);
      key[i] = order_key(k, is_masked(logit[i]));
    }
    if (a.groups > 1) {
      uint32_t* sk = smem_keys + warp * a.experts;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        if (e < a.experts) sk[e] = key[i];
      }
      __syncwarp();
      // lane g scores group g
      uint32_t score = 0;
      if (lane < a.groups) {
        uint32_t first = 0, second = 0;
        for (int e = lane * gsize; e < (lane + 1) * gsize; ++e) {
          const uint32_t v = sk[e];
          second = v > first ? first : (v > second ? v : second);
          first = v > first ? v : first;
        }
        score = first;
        if (a.score == RD_SCORE_SIGMOID && first != 0 && second != 0)
          score = order_key(__fadd_rn(key_of_order(first), key_of_order(second)), false);
      }
      uint32_t kept = 0;
      for (int r = 0; r < a.topk_groups; ++r) {
        const uint32_t best = __reduce_max_sync(kAll, score);
        if (best == 0) break;
        const int g = __ffs(__ballot_sync(kAll, score == best)) - 1;
        kept |= 1u << g;
        if (lane == g) score = 0;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        if (e < a.experts && !((kept >> (e / gsize)) & 1u)) key[i] = 0;
      }
    }
    int my_id = -1;
    for (int k = 0; k < a.topk; ++k) {
      uint32_t mine = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (key[i] > mine) {
          mine = key[i];
          at = i;
        }
      }
      const uint32_t best = __reduce_max_sync(kAll, mine);
      if (best == 0) break;
      const int e = __reduce_min_sync(kAll, mine == best ? lane + 32 * at : 0x7FFFFFFF);
      if (lane == k) my_id = e;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i == e) key[i] = 0;
    }
    const bool there = my_id >= 0;
    const float at = there ? load_logit(row + my_id) : 0.0f;
    float part, total;
    slot_parts<EPL>(a, there, at, logit, part, total);
    if (lane < a.topk) {
      const int64_t o = static_cast<int64_t>(t) * a.topk + lane;
      a.ids[o] = my_id;
      // !(total <= 0) lets a NaN sum through
      a.weights[o] = there && !(total <= 0.0f) ? __fmul_rn(__fdiv_rn(part, total), a.scale) : 0.0f;
    }
  }
}

template <int EPL, class T>
__global__ void __launch_bounds__(kRouteWarps * 32) route_bwd_kernel(const RouteArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t L = tokens_below(a.limit, a.tokens);
  const bool dense = a.score == RD_SCORE_SOFTMAX && !a.renormalize;
  for (int t = blockIdx.x * kRouteWarps + warp; t < L; t += gridDim.x * kRouteWarps) {
    const T* row = static_cast<const T*>(a.logits) + static_cast<int64_t>(t) * a.experts;
    T* out = static_cast<T*>(a.d_logits) + static_cast<int64_t>(t) * a.experts;
    float logit[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      logit[i] = dense && e < a.experts ? load_logit(row + e) : -INFINITY;
    }
    int id = -1;
    float d = 0.0f;
    if (lane < a.topk) {
      const int64_t o = static_cast<int64_t>(t) * a.topk + lane;
      id = a.ids[o];
      if (id >= a.experts) id = -1;
      d = id >= 0 ? a.d_weights[o] : 0.0f;
    }
    const bool there = id >= 0;
    const float at = there ? load_logit(row + id) : 0.0f;
    float part, total;
    slot_parts<EPL>(a, there, at, logit, part, total);
    const float inv = !(total <= 0.0f) ? __fdiv_rn(1.0f, total) : 0.0f;
    const float q = part * inv;
    const float mean = warp_sum(there ? q * d : 0.0f);
    // the rest of the row, then the chosen experts over it
    float top = -INFINITY;
    if (dense) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (!is_masked(logit[i])) top = fmaxf(top, logit[i]);
      top = warp_max(top);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (e >= a.experts) continue;
      float v = 0.0f;
      if (dense && !is_masked(logit[i])) v = -a.scale * (expf(logit[i] - top) * inv) * mean;
      store_logit(out + e, v);
    }
    __syncwarp();
    if (there) {
      float v;
      if (a.score == RD_SCORE_SOFTMAX) v = a.scale * q * (d - mean);
      else v = a.scale * (a.renormalize ? (d - mean) * inv : d) * part * (1.0f - part);
      store_logit(out + id, v);
    }
  }
}

template <class T>
cudaError_t launch_t(const RouteArgs& a, bool bwd, int sms, cudaStream_t stream) {
  const int64_t blocks = (a.tokens + kRouteWarps - 1) / kRouteWarps;
  const int grid = static_cast<int>(blocks < sms * 8 ? blocks : sms * 8);
  const size_t smem = !bwd && a.groups > 1 ? sizeof(uint32_t) * kRouteWarps * a.experts : 0;
  const int epl = (a.experts + 31) / 32;
#define RD_ROUTE(N)                                                                        \
  if (epl <= N) {                                                                          \
    if (bwd) route_bwd_kernel<N, T><<<grid, kRouteWarps * 32, 0, stream>>>(a);             \
    else route_kernel<N, T><<<grid, kRouteWarps * 32, smem, stream>>>(a);                  \
    return cudaGetLastError();                                                             \
  }
  RD_ROUTE(1)
  RD_ROUTE(2)
  RD_ROUTE(4)
  RD_ROUTE(8)
  RD_ROUTE(16)
  RD_ROUTE(32)
#undef RD_ROUTE
  return cudaErrorInvalidValue;
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
