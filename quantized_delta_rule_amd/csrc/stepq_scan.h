// stepq_scan.h -- what the scan's forward and backward kernels share.
#pragma once
#include "stepq_layer.h"

namespace stepq {
namespace lay {

// exp(D A) with a2 = A log2(e).  The hardware's exponential of arguments between -0.01 and 0 is off by -7e-9 of the
// result on average (measured over 2^20 of them; a correct rounding by nothing), and a state that remembers 1,000
// tokens would gather 7e-6 of that.  9.7e-9 more in the argument takes the mean away (below 4e-10); it leaves
// exp(0) at one exactly, so that a step of zero keeps a state's bits, and costs nothing beside the product.
__device__ __forceinline__ float decay(float D, float a2) {
  return __builtin_amdgcn_exp2f(fmaf(D, a2, 9.7e-9f));
}

// The step D of a raw value (softplus: log(1 + exp(v))).  With e = exp(-|v|) and u = 1 + e rounded, log(1 + e) = log(u) +
// (e - (u - 1)) / u, of which the quotient is left out (that takes 2^-24 e / (1 + e) at most, a U of the result): the
// hardware's logarithm by itself would lose a small step behind the one.  Relative error of log(1 + e) measured over
// 1e-8 <= e <= 1: below 2e-7, 5.5e-8 rms; e adds its own.  v = -inf gives a step of zero; NaN passes (by e).
template <int DT>
__device__ __forceinline__ float step_of(int softplus, float v) {
  if (!softplus) return v;
  const float e = exp_minus<DT>(fabsf(v)), u = 1.0f + e;
  return __builtin_amdgcn_fmed3f(v, 0.0f, __builtin_inff()) + fmaf(__builtin_amdgcn_logf(u), 0.693147181f, e - (u - 1.0f));
}
// .. and its derivative, sigmoid(v).
template <int DT>
__device__ __forceinline__ float step_of(int softplus, float v, float& slope) {
  slope = 1.0f;
  if (!softplus) return v;
  const float e = exp_minus<DT>(fabsf(v)), u = 1.0f + e, i = __builtin_amdgcn_rcpf(u);
  slope = v >= 0 ? i : e * i;
  return __builtin_amdgcn_fmed3f(v, 0.0f, __builtin_inff()) + fmaf(__builtin_amdgcn_logf(u), 0.693147181f, e - (u - 1.0f));
}

}  // namespace lay
}  // namespace stepq
