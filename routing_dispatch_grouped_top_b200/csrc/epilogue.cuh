// epilogue.cuh - element-wise math of the products' epilogues.
#pragma once

#include "device.cuh"

namespace moe {

namespace {

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Logistic function with the fast exponential and divide; the quotient's denominator overflows to
// a result of 0 for g -> -inf.
__device__ __forceinline__ float fast_sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// h = silu(g) u.
__device__ __forceinline__ float swiglu(float g, float u) { return __fdividef(g * u, 1.0f + __expf(-g)); }

// Its gradients for dh: dg = dh u s (1 + g (1 - s)), du = dh g s, s = sigma(g).
__device__ __forceinline__ void swiglu_grad(float dh, float g, float u, float& dg, float& du) {
  const float s = fast_sigmoid(g);
  dg = dh * u * s * (1.0f + g * (1.0f - s));
  du = dh * g * s;
}

// Normal distribution function by the Chebyshev fit of erfc of Press et al. (Numerical Recipes,
// section 6.2, fractional error below 1.2e-7 everywhere), Phi(x) = erfc(-x / sqrt 2) / 2.
__device__ __forceinline__ float normal_cdf(float x) {
  const float z = fabsf(x) * 0.70710678f;
  const float t = __fdividef(1.0f, fmaf(0.5f, z, 1.0f));
  float p = 0.17087277f;
  p = fmaf(p, t, -0.82215223f);
  p = fmaf(p, t, 1.48851587f);
  p = fmaf(p, t, -1.13520398f);
  p = fmaf(p, t, 0.27886807f);
  p = fmaf(p, t, -0.18628806f);
  p = fmaf(p, t, 0.09678418f);
  p = fmaf(p, t, 0.37409196f);
  p = fmaf(p, t, 1.00002368f);
  p = fmaf(p, t, -1.26551223f);
  const float e = 0.5f * t * __expf(fmaf(-z, z, p));
  return x < 0.0f ? e : 1.0f - e;
}

// act of `n` values (a moe_act).
template <int n>
__device__ __forceinline__ void activate(float (&v)[n], int act) {
  if (act == MOE_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];  // NaN stays NaN
  } else if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] = __fdividef(v[j], 1.0f + __expf(-v[j]));
  } else if (act == MOE_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] *= normal_cdf(v[j]);
  } else if (act == MOE_ACT_GELU_TANH) {
#pragma unroll
    for (int j = 0; j < n; ++j)
      v[j] *= fast_sigmoid(1.5957691216057308f * (v[j] + 0.044715f * v[j] * v[j] * v[j]));
  }
}

}  // namespace

}  // namespace moe
