// act_math.cuh -- the activations of rd_linear and their derivatives, in f32, two values at a time.
//
// Products and sums are the packed f32x2 forms, an instruction for two values: an elementwise pass over bf16 is
// otherwise bound by instructions before it is by HBM.  exp is the hardware base-2 exponential and 1/x
// the hardware reciprocal, both within a few f32 ulps.
//
// Normal distribution function, from its tail, so that z P(z) keeps its relative precision for z far below zero:
//   P(-|z|) = exp(-z^2 / 2) q(|z|),  q(a) = exp(a^2 / 2) P(-a),  P(|z|) = 1 - P(-|z|).
// q is a polynomial without constant term in t = 1 / (1 + 0.362 a), fitted to it over [0, 14.5] for
// the least relative error (8.5e-7; 1.2e-6 as evaluated in f32); past 13.3 the exponential is taken as 0.
// Logistic: 1 / (1 + exp(-u)), which keeps its relative precision on both sides; below u = -126 ln 2 = -87.34, where it is
// 2^-126, it is 0: the largest value that is lost is silu's there, 1.03e-36, the largest slope the tanh form's, 2.7e-36.
//
// Slopes: arguments are cut to where the slope has reached its limit (0 or 1) exactly, so that infinite z
// give that limit and not 0 * inf; the cuts let NaN through.
#pragma once

#include "../../include/rd_block.h"
#include "glu_math.cuh"

namespace rd {

// ---- packed f32 pairs
__device__ __forceinline__ uint64_t pair_bits(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 bits_pair(uint64_t b) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(b));
  return v;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return bits_pair(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return bits_pair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return bits_pair(r);
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 2^x and 1 / x of the hardware, numbers below 2^-126 to 0 (without that, each would be several instructions)
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// q(a) and exp(-a^2 / 2)
__device__ __forceinline__ void normal_tail(float2 a, float2& q, float2& e) {
  const float2 x = mul2(mul2(a, both(-0.72134752f)), a);  // log2(e) / 2
  e = make_float2(exp2_ftz(x.x), exp2_ftz(x.y));
  const float2 d = fma2(a, both(0.362f), both(1.0f));
  const float2 t = make_float2(rcp_ftz(d.x), rcp_ftz(d.y));
  q = fma2(both(0.0476632722f), t, both(-0.179082657f));
  q = fma2(q, t, both(0.175375615f));
  q = fma2(q, t, both(0.0296722452f));
  q = fma2(q, t, both(0.139128062f));
  q = fma2(q, t, both(0.142743341f));
  q = fma2(q, t, both(0.144500149f));
  q = mul2(q, t);
}

// 1 / (1 + 2^x): the logistic of u for x = -u log2(e)
__device__ __forceinline__ float2 logistic2(float2 x) {
  const float2 d = add2(make_float2(exp2_ftz(x.x), exp2_ftz(x.y)), both(1.0f));
  return make_float2(rcp_ftz(d.x), rcp_ftz(d.y));
}

constexpr float kLog2e = 1.44269504f;
constexpr float kGeluTanhA = 1.59576912f;  // 2 sqrt(2 / pi): (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u))
constexpr float kGeluTanhC = 0.044715f;

template <int ACT>
__device__ __forceinline__ float2 act_value(float2 z) {
  if (ACT == RD_ACT_RELU) return make_float2(max_nan(z.x, 0.0f), max_nan(z.y, 0.0f));
  if (ACT == RD_ACT_GELU) {
    float2 q, e;
    normal_tail(make_float2(fabsf(z.x), fabsf(z.y)), q, e);
    const float2 tail = mul2(q, e), rest = fma2(tail, both(-1.0f), both(1.0f));
    return mul2(z, make_float2(z.x < 0.0f ? tail.x : rest.x, z.y < 0.0f ? tail.y : rest.y));
  }
  if (ACT == RD_ACT_GELU_TANH) {
    const float2 p = fma2(mul2(z, z), both(-kLog2e * kGeluTanhA * kGeluTanhC), both(-kLog2e * kGeluTanhA));
    return mul2(z, logistic2(mul2(z, p)));
  }
  if (ACT == RD_ACT_SILU) return mul2(z, logistic2(mul2(z, both(-kLog2e))));
  return z;
}

template <int ACT>
__device__ __forceinline__ float2 act_slope(float2 z) {
  if (ACT == RD_ACT_RELU)  // NaN stays NaN
    return make_float2(z.x <= 0.0f ? 0.0f : (z.x > 0.0f ? 1.0f : z.x), z.y <= 0.0f ? 0.0f : (z.y > 0.0f ? 1.0f : z.y));
  if (ACT == RD_ACT_GELU) {
    // P(z) + z p(z) = h below zero and 1 - h above, h = exp(-a^2 / 2) (q(a) - a / sqrt(2 pi)), a = |z|
    const float2 a = make_float2(min_nan(fabsf(z.x), 64.0f), min_nan(fabsf(z.y), 64.0f));
    float2 q, e;
    normal_tail(a, q, e);
    const float2 h = mul2(fma2(a, both(-0.39894228f), q), e), rest = fma2(h, both(-1.0f), both(1.0f));
    return make_float2(z.x < 0.0f ? h.x : rest.x, z.y < 0.0f ? h.y : rest.y);
  }
  if (ACT == RD_ACT_GELU_TANH || ACT == RD_ACT_SILU) {
    constexpr bool silu = ACT == RD_ACT_SILU;
    constexpr float cut = silu ? 128.0f : 64.0f;
    z = make_float2(max_nan(min_nan(z.x, cut), -cut), max_nan(min_nan(z.y, cut), -cut));
    float2 s, d;  // the logistic of u, and z du/dz
    if (silu) {
      s = logistic2(mul2(z, both(-kLog2e)));
      d = z;
    } else {
      const float2 zz = mul2(z, z);
      const float2 p = fma2(zz, both(-kLog2e * kGeluTanhA * kGeluTanhC), both(-kLog2e * kGeluTanhA));
      s = logistic2(mul2(z, p));
      d = mul2(z, fma2(zz, both(3.0f * kGeluTanhA * kGeluTanhC), both(kGeluTanhA)));
    }
    const float2 rest = fma2(s, both(-1.0f), both(1.0f));
    return mul2(s, fma2(d, rest, both(1.0f)));
  }
  return both(1.0f);
}

// f(tag) with the run-time activation as the constant tag.value: the switch stands outside the loops
template <int A>
struct ActTag {
  static constexpr int value = A;
};

template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case RD_ACT_RELU: f(ActTag<RD_ACT_RELU>{}); break;
    case RD_ACT_GELU: f(ActTag<RD_ACT_GELU>{}); break;
    case RD_ACT_GELU_TANH: f(ActTag<RD_ACT_GELU_TANH>{}); break;
    case RD_ACT_SILU: f(ActTag<RD_ACT_SILU>{}); break;
    default: f(ActTag<RD_ACT_NONE>{}); break;
  }
}

}  // namespace rd
