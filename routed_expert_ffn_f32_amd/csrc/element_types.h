// Element types of the operators around the layer (COLI_MOE_F32 ...): eight
// consecutive elements at a time between memory and float registers.  Wide
// accesses do not need 16-byte alignment (gfx950 takes global loads and
// stores of any width at element alignment), so rows of any length and
// stride take the same path; only the last, partial eight of a row go one
// element at a time.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "coli_moe.h"

namespace coli {

inline __host__ __device__ size_t type_bytes(int type) {
  return type == COLI_MOE_F32 ? 4 : type == COLI_MOE_BF16 || type == COLI_MOE_F16 ? 2 : 1;
}
inline bool float_type(int type) { return type >= COLI_MOE_F32 && type <= COLI_MOE_F16; }
inline bool byte_type(int type) { return type == COLI_MOE_INT8 || type == COLI_MOE_E4M3; }

__device__ __forceinline__ float from_bf16(uint32_t low16) { return __uint_as_float(low16 << 16); }

// Round to nearest, ties to even; a NaN keeps its sign and stays a NaN.
__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ uint16_t to_f16(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

__device__ __forceinline__ void store1(void *base, int type, int64_t i, float v) {
  if (type == COLI_MOE_F32)
    static_cast<float *>(base)[i] = v;
  else
    static_cast<uint16_t *>(base)[i] = type == COLI_MOE_BF16 ? to_bf16(v) : to_f16(v);
}

// Eight elements as they stand in memory (16-bit types: in lo alone), so that
// loads of several arrays can be in flight before the first is looked at.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
struct Raw8 {
  u32x4 lo, hi;
};

__device__ __forceinline__ u32x4 load16(const char *p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// Elements i .. i + 7.
__device__ __forceinline__ Raw8 load_raw8(const void *base, int type, int64_t i) {
  Raw8 r;
  if (type == COLI_MOE_F32) {
    const char *p = static_cast<const char *>(base) + i * 4;
    r.lo = load16(p);
    r.hi = load16(p + 16);
  } else {
    r.lo = load16(static_cast<const char *>(base) + i * 2);
  }
  return r;
}

// The same, those at n and beyond 0 and not read.  The last, partial eight
// loads its elements from indices held below n, without conditions: a branch
// around each made one wait for the other (a row of 2047 halves: 7 memory
// round trips for every array).
__device__ __forceinline__ Raw8 load_raw8(const void *base, int type, int64_t i, int n) {
  if (n >= 8) return load_raw8(base, type, i);
  Raw8 r = {u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};
  if (n <= 0) return r;
  uint32_t t[7];
  if (type == COLI_MOE_F32) {
    const uint32_t *p = static_cast<const uint32_t *>(base) + i;
#pragma unroll
    for (int j = 0; j < 7; ++j) t[j] = p[min(j, n - 1)];
#pragma unroll
    for (int j = 0; j < 7; ++j) (j < 4 ? r.lo : r.hi)[j & 3] = j < n ? t[j] : 0u;
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(base) + i;
#pragma unroll
    for (int j = 0; j < 7; ++j) t[j] = p[min(j, n - 1)];
#pragma unroll
    for (int j = 0; j < 7; ++j) r.lo[j / 2] |= (j < n ? t[j] : 0u) << (16 * (j & 1));
  }
  return r;
}

__device__ __forceinline__ void unpack8(int type, const Raw8 &r, float (&v)[8]) {
  if (type == COLI_MOE_F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(r.lo[j]);
      v[j + 4] = __uint_as_float(r.hi[j]);
    }
  } else if (type == COLI_MOE_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = from_bf16(r.lo[j]);
      v[2 * j + 1] = __uint_as_float(r.lo[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = (float)__builtin_bit_cast(_Float16, (uint16_t)r.lo[j]);
      v[2 * j + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r.lo[j] >> 16));
    }
  }
}

// v rounded to the 16-bit type (as float32 values; unchanged for F32).
__device__ __forceinline__ void round8(int type, float (&v)[8]) {
  if (type == COLI_MOE_F32) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = type == COLI_MOE_BF16 ? from_bf16(to_bf16(v[j])) : (float)(_Float16)v[j];
}

// Elements i .. i + 7 = v, rounded to the type.
__device__ __forceinline__ void store8(void *base, int type, int64_t i, const float (&v)[8]) {
  if (type == COLI_MOE_F32) {
    __builtin_memcpy(static_cast<float *>(base) + i, v, 32);
    return;
  }
  uint32_t u[4];
  if (type == COLI_MOE_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = to_bf16(v[2 * j]) | ((uint32_t)to_bf16(v[2 * j + 1]) << 16);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = to_f16(v[2 * j]) | ((uint32_t)to_f16(v[2 * j + 1]) << 16);
  }
  __builtin_memcpy(static_cast<uint16_t *>(base) + i, u, 16);
}

// The same, those below n.
__device__ __forceinline__ void store8(void *base, int type, int64_t i, int n, const float (&v)[8]) {
  if (n >= 8) {
    store8(base, type, i, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) store1(base, type, i + j, v[j]);
}

}  // namespace coli
