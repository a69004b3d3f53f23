// The activations of the gated products and their derivatives, in fp32.
#pragma once

#include "common.cuh"

namespace moe {

// All by forms that keep their relative precision where the activation dies out (a
// sum 1 + erf or 1 + tanh loses it): Phi(g) = erfc(-g / sqrt 2) / 2 by the Chebyshev fit of
// Press et al., Numerical Recipes, section 6.2 (fractional error below 1.2e-7 for every
// argument; CUDA's erfcf bounded the elementwise backward: 2043 x 1537 elements 24 us),
// and the form by tanh
// is g times the logistic function of 2 sqrt(2 / pi) (g + 0.044715 g^3).  The hardware's
// exponential as in the layer's SwiGLU: every use is rounded to 16 bits.
constexpr float kTanhSlope = 1.5957691216057308f, kTanhCube = 0.044715f;

MOE_DEV float erfc_fit(float x) {
  const float z = fabsf(x), t = __fdividef(1.0f, fmaf(0.5f, z, 1.0f));
  float p = fmaf(t, 0.17087277f, -0.82215223f);
  p = fmaf(t, p, 1.48851587f);
  p = fmaf(t, p, -1.13520398f);
  p = fmaf(t, p, 0.27886807f);
  p = fmaf(t, p, -0.18628806f);
  p = fmaf(t, p, 0.09678418f);
  p = fmaf(t, p, 0.37409196f);
  p = fmaf(t, p, 1.00002368f);
  p = fmaf(t, p, -1.26551223f);
  const float tail = t * __expf(fmaf(-z, z, p));
  return x >= 0.f ? tail : 2.0f - tail;
}

// act(g).
template <int ACT>
MOE_DEV float act_value(float g) {
  if constexpr (ACT == MOE_ACT_SILU) return silu(g);
  if constexpr (ACT == MOE_ACT_GELU) return 0.5f * g * erfc_fit(g * -0.70710678118654752f);
  if constexpr (ACT == MOE_ACT_GELU_TANH) return g * sigmoidf(kTanhSlope * g * (1.0f + kTanhCube * g * g));
  return g <= 0.f ? 0.f : g;  // NaN stays
}

// act(g) and act'(g).
template <int ACT>
MOE_DEV void act_slope(float g, float &value, float &slope) {
  if constexpr (ACT == MOE_ACT_SILU) {
    const float s = sigmoidf(g);
    value = g * s;
    slope = s * (1.0f + g * (1.0f - s));
  } else if constexpr (ACT == MOE_ACT_GELU) {
    const float cdf = 0.5f * erfc_fit(g * -0.70710678118654752f);
    value = g * cdf;
    slope = cdf + g * __expf(-0.5f * g * g) * 0.39894228040143268f;
  } else if constexpr (ACT == MOE_ACT_GELU_TANH) {
    // s is 0 or 1 long before g^2 = 10^4; where g^2 itself overflows, 0 * inf would be NaN
    const float q = kTanhCube * fminf(g * g, 1e4f), s = sigmoidf(kTanhSlope * g * (1.0f + q));
    value = g * s;
    slope = s + value * (1.0f - s) * kTanhSlope * (1.0f + 3.0f * q);
  } else {
    value = g <= 0.f ? 0.f : g;
    slope = g <= 0.f ? 0.f : 1.f;
  }
}

}  // namespace moe
