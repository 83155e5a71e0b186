// Scalar functions of the operators around the layer, float32.
#pragma once

#include <hip/hip_runtime.h>

namespace coli {

// exp(x) for x <= 0 (Cody and Waite): x = n ln 2 + r with ln 2 in two parts (n r exact enough
// that r keeps full precision), 2^(r / ln 2) on the transcendental unit, n
// through the exponent.  -Inf gives 0.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2e = 1.44269504f, kLn2Hi = 0.693359375f, kLn2Lo = -2.12194440e-4f;
  x = fmaxf(x, -110.0f);  // below: 0 anyway (a NaN becomes 0 here)
  const float n = rintf(x * kLog2e);
  const float r = __builtin_fmaf(-n, kLn2Lo, __builtin_fmaf(-n, kLn2Hi, x));
  return __builtin_ldexpf(__builtin_amdgcn_exp2f(r * kLog2e), (int)n);
}

// sigma(v) = 1 / (1 + exp(-v)), without overflow on either side.
__device__ __forceinline__ float sigmoid(float v) {
  const float a = exp_neg(-fabsf(v));
  return (v >= 0.0f ? 1.0f : a) * (1.0f / (1.0f + a));
}

}  // namespace coli
