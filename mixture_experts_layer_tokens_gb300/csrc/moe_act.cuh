// Activations and their slopes in fp32, shared by the linear and the activation kernels.
#pragma once
#include "moe_vec.cuh"

namespace moe {
namespace {

// 1 / (1 + exp(-x)) within 2^-21 (the exponential's error is weighed by at most 0.65 / (2 + 1.2 |x|)),
// and 0 or 1 where exp overflows or vanishes.
__device__ __forceinline__ float fast_sigmoid(float x) { return fast_rcp(1.0f + fast_exp(-x)); }

// sqrt(2/pi) (z + 0.044715 z^3): (1 + tanh(u)) / 2 is the sigmoid of 2 u
__device__ __forceinline__ float gelu_u(float z) { return 0.79788456f * z * fmaf(0.044715f * z, z, 1.0f); }

// The normal distribution below -x, x >= 0, with e = exp(-x^2 / 2): e t P(t), t = 1 / (1 + 0.305 x) (the form of
// Hastings' approximations of erf), P of degree 7 fitted to erfcx(x / sqrt 2) / (2 t) for the least largest relative
// error on [0, 14]: 0.8 2^-23, in fp32 with e and 1 / x as above within (0.85 x^2 + 6) 2^-23 of the value
// where it does not vanish (x < 13.2).  GELU from it keeps its digits below 0, where z/2 (1 + erf)
// cancels (4 % of the value at -5), and the gradient shares e.  8192 x 4096 over 512 with a full epilogue: 89
// us, by erfcf 133, by 1 + erff 100.
__device__ __forceinline__ float normal_below(float x, float e) {
  const float t = fast_rcp(fmaf(0.305f, x, 1.0f));
  float p = 0.0367012769f;
  p = fmaf(p, t, -0.152997345f);
  p = fmaf(p, t, 0.18573311f);
  p = fmaf(p, t, -0.0379923917f);
  p = fmaf(p, t, 0.121030286f);
  p = fmaf(p, t, 0.103418142f);
  p = fmaf(p, t, 0.122467272f);
  p = fmaf(p, t, 0.121639699f);
  return p * t * e;
}

__device__ __forceinline__ float act_fwd(float z, int act) {
  switch (act) {
    case MOE_LINEAR_SILU: return z * fast_sigmoid(z);
    case MOE_LINEAR_GELU: {
      const float x = fminf(fabsf(z), 16.f);  // (the tail is 0 there)
      return fmaf(-x, normal_below(fabsf(z), fast_exp(-0.5f * x * x)), fmaxf(z, 0.f));
    }
    case MOE_LINEAR_GELU_TANH: return z * fast_sigmoid(2.0f * gelu_u(z));
  }
  return z;
}

// The slopes are 1 or 0 to fp32 beyond |z| = 128 (silu) and 16; c, z kept to that range, goes into the factors
// that grow, so that they stay finite where the one that vanishes is 0 (z = 1e20, or the infinity that a
// sum became in 16 bits).  A NaN comes through the sigmoid or the tail of z itself.
__device__ __forceinline__ float act_grad(float z, int act) {
  const float c = fminf(fmaxf(z, act == MOE_LINEAR_SILU ? -128.f : -16.f), act == MOE_LINEAR_SILU ? 128.f : 16.f);
  switch (act) {
    case MOE_LINEAR_SILU: {
      const float q = fast_sigmoid(z);
      return q * fmaf(c, 1.0f - q, 1.0f);
    }
    case MOE_LINEAR_GELU: {
      const float e = fast_exp(-0.5f * c * c), below = normal_below(fabsf(z), e);
      return fmaf(c * 0.39894228f, e, z < 0.f ? below : 1.0f - below);
    }
    case MOE_LINEAR_GELU_TANH: {
      const float q = fast_sigmoid(2.0f * gelu_u(z));
      // z q (1 - q) 2 u'
      return fmaf(c * q * (1.0f - q), 1.59576912f * fmaf(0.134145f * c, c, 1.0f), q);
    }
  }
  return 1.0f;
}

}  // namespace
}  // namespace moe
