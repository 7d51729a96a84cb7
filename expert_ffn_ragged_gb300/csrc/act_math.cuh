// act_math.cuh -- the activations of rd_linear and their derivatives, in f32.
//
// exp comes from the hardware base-2 exponential and 1/x from the hardware reciprocal (glu_math.cuh), both
// within a few f32 ulps.  The normal distribution function is taken from its tail, so that
// z P(z) keeps its relative precision for z far below zero:
//   P(-|z|) = exp(-z^2 / 2) q(|z|),  q(a) = exp(a^2 / 2) P(-a),  P(|z|) = 1 - P(-|z|).
// q is a polynomial without constant term in t = 1 / (1 + 0.3 a), fitted to it over [0, 14.5] for
// the least relative error (1.6e-7; 5e-7 as evaluated in f32); past 14.5 the exponential is below
// f32's smallest number.
//
// Derivatives have the form s + z b with b going to zero faster than 1 / z: where b is 0 the product is left
// out, so that infinite z give the limits (0 or 1) and not 0 * inf.
#pragma once

#include "../../include/rd_block.h"
#include "glu_math.cuh"

namespace rd {

// P(z), and e = exp(-z^2 / 2)
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float a = fabsf(z);
  e = exp2_approx(-0.72134752f * z * z);  // log2(e) / 2
  const float t = rcp_approx(fmaf(0.3f, a, 1.0f));
  float q = 0.0354249f;
  q = fmaf(q, t, -0.15616337f);
  q = fmaf(q, t, 0.20456536f);
  q = fmaf(q, t, -0.05204196f);
  q = fmaf(q, t, 0.12769598f);
  q = fmaf(q, t, 0.10017468f);
  q = fmaf(q, t, 0.12071234f);
  q = fmaf(q, t, 0.11963199f);
  const float tail = q * t * e;
  return z < 0.0f ? tail : 1.0f - tail;
}

constexpr float kGeluTanhA = 1.59576912f;  // 2 sqrt(2 / pi): (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u))
constexpr float kGeluTanhC = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == RD_ACT_RELU) return z <= 0.0f ? 0.0f : z;  // NaN stays NaN
  if (ACT == RD_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  if (ACT == RD_ACT_GELU_TANH || ACT == RD_ACT_SILU) {
    const float u = ACT == RD_ACT_SILU ? z : kGeluTanhA * z * fmaf(kGeluTanhC * z, z, 1.0f);
    float sig, om;
    sigmoid_two_sided(u, sig, om);
    return z * sig;
  }
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == RD_ACT_RELU) return z <= 0.0f ? 0.0f : (z > 0.0f ? 1.0f : z);  // NaN stays NaN
  if (ACT == RD_ACT_GELU) {
    float e;
    const float p = normal_cdf(z, e);
    return e == 0.0f ? p : fmaf(z, 0.39894228f * e, p);  // 1 / sqrt(2 pi)
  }
  if (ACT == RD_ACT_GELU_TANH || ACT == RD_ACT_SILU) {
    const bool silu = ACT == RD_ACT_SILU;
    const float zz = kGeluTanhC * z * z;
    const float u = silu ? z : kGeluTanhA * z * (1.0f + zz);
    float sig, om;
    sigmoid_two_sided(u, sig, om);
    const float bell = sig * om;
    const float du = silu ? z : kGeluTanhA * z * fmaf(3.0f, zz, 1.0f);
    return bell == 0.0f ? sig : fmaf(du, bell, sig);
  }
  return 1.0f;
}

// f(std::integral_constant-like tag) for a run-time activation: the switch stands outside the loops
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
