// What the kernels of coli_moe_linear share: the products of 16-byte operand
// pieces on the matrix cores, and the epilogue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "coli_moe.h"
#include "element_types.h"
#include "lds_dma.h"
#include "scalar_math.h"
#include "wave.h"

namespace coli {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Operand types: a 16-byte piece of a row in every lane is one operand of an
// MFMA (e4m3: of two).  The matrix cores sum over K in any order the two
// operands agree on, so both take the same pieces of their rows and the layout
// within K does not matter.  int8 products accumulate exactly in int32, at
// twice the 16-bit rate, the others in float32.
template <int TYPE>
struct Operand;

template <>
struct Operand<COLI_MOE_BF16> {
  typedef f32x16 Acc32;
  typedef f32x4 Acc16;
  static __device__ __forceinline__ Acc32 mma(uint4 a, uint4 b, Acc32 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                   c, 0, 0, 0);
  }
  static __device__ __forceinline__ Acc16 mma(uint4 a, uint4 b, Acc16 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                   c, 0, 0, 0);
  }
};

template <>
struct Operand<COLI_MOE_F16> {
  typedef f32x16 Acc32;
  typedef f32x4 Acc16;
  static __device__ __forceinline__ Acc32 mma(uint4 a, uint4 b, Acc32 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                  0, 0, 0);
  }
  static __device__ __forceinline__ Acc16 mma(uint4 a, uint4 b, Acc16 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                  0, 0, 0);
  }
};

template <>
struct Operand<COLI_MOE_INT8> {
  typedef i32x16 Acc32;
  typedef i32x4 Acc16;
  static __device__ __forceinline__ Acc32 mma(uint4 a, uint4 b, Acc32 c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0,
                                                 0, 0);
  }
  static __device__ __forceinline__ Acc16 mma(uint4 a, uint4 b, Acc16 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0,
                                                 0, 0);
  }
};

// e4m3 on the 16-bit matrix cores: every code is a half exactly, so sums are
// float32 sums.  (The 8-bit float MFMAs add each group of 8 products with
// about 15 bits below the largest of them: measured, 2^16 + 7 * 1 within a
// group gives 2^16, and the worst error of 64 random products was 2^-12.3 of
// the largest.)
template <>
struct Operand<COLI_MOE_E4M3> {
  typedef f32x16 Acc32;
  typedef f32x4 Acc16;
  // codes 8 h .. 8 h + 7 of a piece
  static __device__ __forceinline__ f16x8 halves(const uint4 &v, int h) {
    const int lo = (int)(h ? v.z : v.x), hi = (int)(h ? v.w : v.y);
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const auto c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return f16x8{(_Float16)a[0], (_Float16)a[1], (_Float16)b[0], (_Float16)b[1],
                 (_Float16)c[0], (_Float16)c[1], (_Float16)d[0], (_Float16)d[1]};
  }
  static __device__ __forceinline__ Acc32 mma(uint4 a, uint4 b, Acc32 c) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(halves(a, 0), halves(b, 0), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(halves(a, 1), halves(b, 1), c, 0, 0, 0);
  }
  static __device__ __forceinline__ Acc16 mma(uint4 a, uint4 b, Acc16 c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(halves(a, 0), halves(b, 0), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(halves(a, 1), halves(b, 1), c, 0, 0, 0);
  }
};

// 16 zero bytes: where the copies past a row's end come from.
__device__ const uint4 kZeroPiece = {0u, 0u, 0u, 0u};

// Elements i .. i + 7 of an array as float32; WHOLE: all of them exist, else
// those at i + n and beyond are 0 and not read.
template <bool WHOLE>
__device__ __forceinline__ void fetch8(const void *base, int type, int64_t i, int n, float (&v)[8]) {
  unpack8(type, WHOLE ? load_raw8(base, type, i) : load_raw8(base, type, i, n), v);
}

// v[j] *= sx w[j], the sum times the row's scale first: the product of two
// scales alone may leave float32's range where the result does not (two of
// 1e-22 on a sum of 2^30).  A sum other than 0 lies in 2^-18 .. 2^34, so with
// sx in 2^-90 .. 2^90 the first product is a normal float32, whatever w is;
// rows of other scales are multiplied in float64.
__device__ __forceinline__ void scale8(float (&v)[8], float sx, const float (&w)[8]) {
  const float size = fabsf(sx);
  if ((size < 0x1p-90f && size > 0.0f) || size > 0x1p+90f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)((double)v[j] * sx * w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * sx * w[j];
  }
}

// The epilogue up to the residual of 8 neighbouring outputs (row m, columns n
// .. n + 7): v = the products' sums (up: those of the up rows, SwiGLU only),
// float32.  WHOLE: n + 7 < a.n.
template <bool WHOLE>
__device__ __forceinline__ void activate8(const coli_moe_linear_t &a, int m, int n, float (&v)[8], float (&up)[8]) {
  const int cnt = a.n - n;
  const bool gated = a.act == COLI_MOE_ACT_SWIGLU;
  float w[8];
  if (a.x_scale) {
    const float sx = a.x_scale[m];
    fetch8<WHOLE>(a.w_scale, COLI_MOE_F32, n, cnt, w);
    scale8(v, sx, w);
    if (gated) {
      fetch8<WHOLE>(a.w_scale, COLI_MOE_F32, (int64_t)a.n + n, cnt, w);
      scale8(up, sx, w);
    }
  }
  if (a.bias) {
    fetch8<WHOLE>(a.bias, a.bias_type, n, cnt, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += w[j];
    if (gated) {
      fetch8<WHOLE>(a.bias, a.bias_type, (int64_t)a.n + n, cnt, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) up[j] += w[j];
    }
  }
  switch (a.act) {
    case COLI_MOE_ACT_RELU:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];  // keeps a NaN
      break;
    case COLI_MOE_ACT_SILU:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * sigmoid(v[j]);
      break;
    case COLI_MOE_ACT_GELU:
#pragma nounroll
      for (int j = 0; j < 8; ++j) {  // a long function: one copy of it, on rotating values
        const float y = 0.5f * v[0] * erfcf(v[0] * -0.70710678f);
#pragma unroll
        for (int q = 0; q < 7; ++q) v[q] = v[q + 1];
        v[7] = y;
      }
      break;
    case COLI_MOE_ACT_GELU_TANH:  // tanh(u) = 2 sigma(2 u) - 1
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = v[j] * sigmoid(1.59576912f * (v[j] + 0.044715f * v[j] * v[j] * v[j]));
      break;
    case COLI_MOE_ACT_SWIGLU:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * sigmoid(v[j]) * up[j];
      break;
    default: break;
  }
}

// The rest of it: adds the residual (as loaded) and stores.
template <bool WHOLE>
__device__ __forceinline__ void store_out8(const coli_moe_linear_t &a, int m, int n, float (&v)[8], const Raw8 &res) {
  if (a.residual) {
    float r[8];
    unpack8(a.out_type, res, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
  }
  if (WHOLE)
    store8(a.out, a.out_type, (int64_t)m * a.ldo + n, v);
  else
    store8(a.out, a.out_type, (int64_t)m * a.ldo + n, a.n - n, v);
}

}  // namespace coli
