// Scalar functions of the operators around the layer, float32.
#pragma once

#include <hip/hip_runtime.h>

namespace coli {

// exp(x) for x <= 0: 2^t on the transcendental unit with t = x / ln 2 rounded,
// corrected by the rounding error of t (the remainder of the product, and the
// part of 1 / ln 2 that float32 leaves off): within about 2^-22.  -Inf gives 0,
// a NaN stays one, results below 2^-126 are 0.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;  // 1 / ln 2 = kHi + kLo
  x = __builtin_elementwise_maximum(x, -110.0f);  // below: 0 anyway; keeps a NaN
  const float t = x * kHi;
  const float rest = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -t));
  const float r = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(r * kLn2, rest, r);
}

// sigma(v) = 1 / (1 + exp(-v)), without overflow on either side.
__device__ __forceinline__ float sigmoid(float v) {
  const float a = exp_neg(-fabsf(v));
  return (v >= 0.0f ? 1.0f : a) * __builtin_amdgcn_rcpf(1.0f + a);
}

}  // namespace coli
