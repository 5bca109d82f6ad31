// stepq_scan.h -- what the scan's forward and backward kernels share.
#pragma once
#include "stepq_layer.h"

namespace stepq {
namespace lay {

constexpr float kLog2e = 1.44269504f;

// exp(D A) with a2 = A log2(e).  The hardware's exponential of arguments between -0.01 and 0 is off by -7e-9 of the
// result on average (measured over 2^20 of them; a correct rounding by nothing), and a state that remembers 1,000
// tokens would gather 7e-6 of that.  9.7e-9 more in the argument takes the mean away (below 4e-10); it leaves
// exp(0) at one exactly, so that a step of zero keeps a state's bits, and costs nothing beside the product.
__device__ __forceinline__ float decay(float D, float a2) {
  return __builtin_amdgcn_exp2f(fmaf(D, a2, 9.7e-9f));
}

// log(1 + e) for 0 <= e <= 1, relative error below 2^-22: twice the inverse hyperbolic tangent of s = e / (2 + e) <= 1/3
// by its series s (1 + s^2/3 + s^4/5 + ..), whose first term left out is s^14/15 < 2^-26 of the whole.
__device__ __forceinline__ float log1p_unit(float e) {
  const float d = 2.0f + e, r = __builtin_amdgcn_rcpf(d);
  float s = e * r;
  s = fmaf(fmaf(-s, d, e), r, s);
  const float q = s * s;
  float p = fmaf(q, 1.0f / 13, 1.0f / 11);
  p = fmaf(p, q, 1.0f / 9);
  p = fmaf(p, q, 1.0f / 7);
  p = fmaf(p, q, 1.0f / 5);
  p = fmaf(p, q, 1.0f / 3);
  p = fmaf(p, q, 1.0f);
  return (s + s) * p;
}

// exp(v) for v <= 0 (0 below -150; NaN too: the caller looks for it).  The product with log2(e) is taken with its rounding error: a step of exp(-10) rounded
// at its argument alone would be off by 2^-21.
__device__ __forceinline__ float exp_neg(float v) {
  v = fmaxf(v, -150.0f);
  const float p = v * kLog2e;
  const float r = fmaf(v, kLog2e, -p) + v * 1.92596303e-8f;  // log2(e) - kLog2e
  const float x = __builtin_amdgcn_exp2f(p);
  return fmaf(x, r * 0.693147181f, x);
}

// The step D of a raw value, and its derivative (softplus: log(1 + exp(v)), sigmoid(v)).
__device__ __forceinline__ float step_of(int softplus, float v, float& slope) {
  slope = 1.0f;
  if (!softplus) return v;
  const float e = exp_neg(-fabsf(v));
  const float i = __builtin_amdgcn_rcpf(1.0f + e);
  slope = v >= 0 ? i : e * i;
  return v == v ? fmaxf(v, 0.0f) + log1p_unit(e) : v;
}

}  // namespace lay
}  // namespace stepq
