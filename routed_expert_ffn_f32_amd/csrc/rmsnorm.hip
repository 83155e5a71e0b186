// Residual addition with the root-mean-square norm (coli_moe_rmsnorm):
//
//   s = x + residual,  y = (s r) weight,  r = 1 / sqrt(sum(s^2) / h + eps),
//
// and, for 8-bit outputs, scale = max|y| / Q and codes round(y / scale) per
// row or per group of columns.
//
// Bound by bytes: every element is read once, kept in registers across the
// reductions and written once (about 20 float32 operations and two float64
// ones an element, against 6 to 13 bytes of HBM traffic).  A thread holds
// NCH pieces of 8 columns, so a row is one pass whatever its length.
//
// The sum of squares is kept in float64: squares of float32 values are then
// exact to 2^-53 of the sum, and r, rounded once to float32, is the same
// number for every split of the row over threads, so that all launch shapes
// below give the same bits.
#include "element_types.h"
#include "internal.h"
#include "wave.h"

namespace coli {
namespace {

constexpr int kVec = 8;  // columns of one piece

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int m = LANES / 2; m; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// Codes of one piece: round(y / scale) to the nearest, ties to even.
__device__ __forceinline__ uint64_t codes8(const float (&y)[kVec], float scale, bool e4m3) {
  uint32_t w[2] = {0u, 0u};
  if (!(scale > 0.0f)) return 0;
  const float q = e4m3 ? 448.0f : 127.0f;
  float v[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) v[j] = fminf(fmaxf(y[j] / scale, -q), q);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (e4m3) {
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
      p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], p, true);
      w[h] = (uint32_t)p;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[h] |= ((uint32_t)(int)rintf(v[4 * h + j]) & 0xFFu) << (8 * j);
    }
  }
  return w[0] | ((uint64_t)w[1] << 32);
}

// WAVES waves hold one row, NCH pieces a thread.  WAVES == 1: four rows a
// workgroup, one per wave, no barrier.
template <int WAVES, int NCH>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void rmsnorm_kernel(coli_moe_rmsnorm_t a) {
  constexpr int kThreads = 64 * WAVES;
  __shared__ double sum_of[WAVES];
  __shared__ float max_of[WAVES];
  const int wave = WAVES == 1 ? 0 : (int)(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int tid = WAVES == 1 ? lane : (int)threadIdx.x;
  const int64_t row = WAVES == 1 ? (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (row >= a.rows) return;  // whole waves; only WAVES == 1 has such rows
  const int h = a.hidden;

  float s[NCH][kVec];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = kVec * (i * kThreads + tid);
    load8(a.x, a.x_type, row * a.x_stride + c, h - c, s[i]);
  }
  if (a.residual) {
    float r[NCH][kVec];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = kVec * (i * kThreads + tid);
      load8(a.residual, a.residual_type, row * a.residual_stride + c, h - c, r[i]);
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[i][j] += r[i][j];
      round8(a.residual_type, s[i]);
    }
  }
  float w[NCH][kVec];
  if (a.weight) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = kVec * (i * kThreads + tid);
      load8(a.weight, a.weight_type, c, h - c, w[i]);
    }
  }
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = kVec * (i * kThreads + tid);
      store8(a.residual_out, a.residual_type, row * a.residual_out_stride + c, h - c, s[i]);
    }
  }

  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) sum = __builtin_fma((double)s[i][j], (double)s[i][j], sum);
  sum = wave_sum64(sum);
  if constexpr (WAVES > 1) {
    if (lane == 0) sum_of[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) sum += sum_of[i];
  }
  const float r = (float)(1.0 / sqrt(sum / (double)h + (double)a.eps));
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      s[i][j] *= r;
      if (a.weight) s[i][j] *= w[i][j];
    }

  if (a.out_type <= COLI_MOE_F16) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = kVec * (i * kThreads + tid);
      store8(a.out, a.out_type, row * a.out_stride + c, h - c, s[i]);
    }
    return;
  }

  // 8 bits: the largest magnitude of the row or of each group (pieces past
  // the row's end hold zeros), then the codes
  const bool e4m3 = a.out_type == COLI_MOE_E4M3;
  const float q = e4m3 ? 448.0f : 127.0f;
  float m[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    m[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) m[i] = fmaxf(m[i], fabsf(s[i][j]));
  }
  if (a.group == 0) {
    float all = m[0];
#pragma unroll
    for (int i = 1; i < NCH; ++i) all = fmaxf(all, m[i]);
    all = lanes_max<64>(all);
    if constexpr (WAVES > 1) {
      if (lane == 0) max_of[wave] = all;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < WAVES; ++i) all = fmaxf(all, max_of[i]);
    }
    const float scale = all / q;
    if (tid == 0) a.scales[row * a.scales_stride] = scale;
#pragma unroll
    for (int i = 0; i < NCH; ++i) m[i] = scale;
  } else {
    // a group's pieces sit in 8 or 16 neighbouring lanes
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      m[i] = (a.group == 64 ? lanes_max<8>(m[i]) : lanes_max<16>(m[i])) / q;
      const int c = kVec * (i * kThreads + tid);
      if (c < h && c % a.group == 0) a.scales[row * a.scales_stride + c / a.group] = m[i];
    }
  }
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = kVec * (i * kThreads + tid);
    if (c >= h) continue;
    const uint64_t codes = codes8(s[i], m[i], e4m3);
    uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.out_stride + c;
    if (h - c >= kVec)
      __builtin_memcpy(out, &codes, 8);
    else
      for (int j = 0; j < h - c; ++j) out[j] = (uint8_t)(codes >> (8 * j));
  }
}

template <int WAVES, int NCH>
hipError_t launch_shape(const coli_moe_rmsnorm_t &a, hipStream_t s) {
  const int rows = WAVES == 1 ? (a.rows + 3) / 4 : a.rows;
  return launch(rmsnorm_kernel<WAVES, NCH>, dim3(rows), dim3(WAVES == 1 ? 256 : 64 * WAVES), 0, s, a);
}

}  // namespace

hipError_t launch_rmsnorm(const coli_moe_rmsnorm_t &a, hipStream_t s) {
  const int pieces = (a.hidden + kVec - 1) / kVec;
  if (pieces <= 64) return launch_shape<1, 1>(a, s);
  if (pieces <= 128) return launch_shape<1, 2>(a, s);
  if (pieces <= 256) return launch_shape<4, 1>(a, s);
  if (pieces <= 512) return launch_shape<4, 2>(a, s);
  if (pieces <= 768) return launch_shape<4, 3>(a, s);
  if (pieces <= 1024) return launch_shape<16, 1>(a, s);
  if (pieces <= 2048) return launch_shape<16, 2>(a, s);
  return launch_shape<16, 4>(a, s);
}

}  // namespace coli
