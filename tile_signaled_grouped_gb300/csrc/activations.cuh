// The activations of the operators (linear.cu, gated.cu) and their derivatives, in fp32.
#pragma once

#include "ops_common.cuh"

#if defined(__CUDACC__)

namespace moe {

__device__ __forceinline__ float fast_sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

constexpr float kGeluC0 = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluC1 = 0.044715f;

// The normal distribution: returns (1 + erf(z / sqrt(2))) / 2, and in *e exp(-z^2 / 2). The
// side of 0 that z is on has the tail q = erfc(|z| / sqrt(2)) / 2 = e t R(t), t = 1 / (1 + 0.44 |z| /
// sqrt(2)): without the exponential it falls only as 1 / |z|, and R is a polynomial fitted to it over
// |z| < 14, where e leaves fp32, with the largest relative error as small as degree 7 allows
// (1.9e-7; least squares reweighted by the errors, Lawson's method). So nothing cancels below 0,
// where 1 + erf keeps multiples of 6e-8 only (4 % of gelu at -5). Within (1.5 z^2 + 25) 2^-24 of
// itself: three roundings of the exponent, and 25 half steps for the rest. 4096 x 4096 x 1024
// with this gelu takes 42 us, 47 by erff, 67 by erfcf.
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  float t, x;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(fabsf(z), 0.44f * 0.7071067811865476f, 1.0f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(z * z * -0.7213475204444817f));  // log2(e) / 2
  float r = 0.035597959f;
  r = fmaf(r, t, -0.13891378f);
  r = fmaf(r, t, 0.14823441f);
  r = fmaf(r, t, -0.0099838804f);
  r = fmaf(r, t, 0.10784631f);
  r = fmaf(r, t, 0.10867608f);
  r = fmaf(r, t, 0.12443229f);
  r = fmaf(r, t, 0.12411071f);
  const float q = r * t * x;
  *e = x;
  return z < 0.f ? q : 1.0f - q;
}

// act(z). 0.5 (1 + tanh u) is the sigmoid of 2u. The fast exponential of v is within
// (2 + 1.2 |v|) 2^-23 of itself (1e-6 at 6, 1e-5 at 80) and the fast division within 2^-22, far
// below half a step of a 16-bit result; an fp32 result is off by that. Sigmoids below 2^-126 are 0.
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if (ACT == MOE_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays
  if (ACT == MOE_ACT_GELU) {
    float e;
    return z * normal_cdf(z, &e);
  }
  if (ACT == MOE_ACT_GELU_TANH) return z * fast_sigmoid(2.0f * kGeluC0 * (z + kGeluC1 * z * z * z));
  if (ACT == MOE_ACT_SILU) return z * fast_sigmoid(z);
  return z;
}
// act'(z). z is kept where it makes no infinities times zero: past 30 the derivatives are 1 to
// the last bit, and below -30 0 in fp32, but for silu's, z exp(z), which is below 1e-36 only
// from -88 on and 0 here. NaN stays (relu's derivative there is 0).
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if (ACT == MOE_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  constexpr float kLow = ACT == MOE_ACT_SILU ? -100.f : -30.f;
  z = z > 30.f ? 30.f : z < kLow ? kLow : z;
  if (ACT == MOE_ACT_GELU) {
    float e;
    const float p = normal_cdf(z, &e);
    return fmaf(z * 0.3989422804014327f, e, p);  // 1 / sqrt(2 pi)
  }
  if (ACT == MOE_ACT_GELU_TANH) {
    const float q = fast_sigmoid(2.0f * kGeluC0 * (z + kGeluC1 * z * z * z));
    return q + z * q * (1.0f - q) * (2.0f * kGeluC0) * (1.0f + 3.0f * kGeluC1 * z * z);
  }
  if (ACT == MOE_ACT_SILU) {
    const float q = fast_sigmoid(z);
    return q * (1.0f + z * (1.0f - q));
  }
  return 1.f;
}

// act(z), and in *d act'(z), as act_of and act_grad have them (bit for bit: where act_grad keeps z
// inside its limits, what it takes of z there is 0 or 1 on both sides of them): the exponential is shared.
template <int ACT>
__device__ __forceinline__ float act_both(float z, float* d) {
  if (ACT == MOE_ACT_SILU || ACT == MOE_ACT_GELU || ACT == MOE_ACT_GELU_TANH) {
    constexpr float kLow = ACT == MOE_ACT_SILU ? -100.f : -30.f;
    const float v = z > 30.f ? 30.f : z < kLow ? kLow : z;
    if (ACT == MOE_ACT_GELU) {
      float e;
      const float p = normal_cdf(z, &e);
      *d = fmaf(v * 0.3989422804014327f, e, p);
      return z * p;
    }
    if (ACT == MOE_ACT_GELU_TANH) {
      const float q = fast_sigmoid(2.0f * kGeluC0 * (z + kGeluC1 * z * z * z));
      *d = q + v * q * (1.0f - q) * (2.0f * kGeluC0) * (1.0f + 3.0f * kGeluC1 * v * v);
      return z * q;
    }
    const float q = fast_sigmoid(z);
    *d = q * (1.0f + v * (1.0f - q));
    return z * q;
  }
  *d = act_grad<ACT>(z);
  return act_of<ACT>(z);
}

}  // namespace moe

#endif  // __CUDACC__
