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
// NCH pieces of 8 columns, so a row is one pass whatever its length.  4096 x
// 6144: bf16 with a bf16 residual 41.7 us (4.8 TB/s; a copy of as many bytes
// runs at 5.1 to 5.2), int8 from bf16 with a float32 residual 56 us (4.9
// TB/s).  One row of 6144 takes 3.2 us, of which a launch is about 2: two
// memory round trips and the reductions.
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

// 1 / sqrt(m), m > 0: the instruction's estimate (about 2^-24) and two Newton
// steps, far below the float32 it is rounded to.
__device__ __forceinline__ double rsqrt64(double m) {
  double y = __builtin_amdgcn_rsq(m);
  y = __builtin_fma(0.5 * y, __builtin_fma(-m * y, y, 1.0), y);
  return __builtin_fma(0.5 * y, __builtin_fma(-m * y, y, 1.0), y);
}

// Codes of one piece: round(y / scale) to the nearest, ties to even.  With
// the correctly rounded reciprocal, one remainder step gives the correctly
// rounded quotient (Markstein), 3 operations where a division takes 10; below
// kTiny the reciprocal or the remainder could leave float32's range.
__device__ __forceinline__ uint64_t codes8(const float (&y)[kVec], float scale, bool e4m3) {
  constexpr float kTiny = 0x1p-60f, kHuge = 0x1p+100f;
  if (!(scale > 0.0f && scale < __builtin_inff())) return 0;
  const float q = e4m3 ? 448.0f : 127.0f, inv = 1.0f / scale;
  const bool divide = !(scale >= kTiny && scale <= kHuge);
  float v[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    float t = y[j] * inv;
    t = __builtin_fmaf(__builtin_fmaf(-t, scale, y[j]), inv, t);
    if (divide) t = y[j] / scale;
    v[j] = __builtin_amdgcn_fmed3f(t, -q, q);
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (e4m3) {
#pragma unroll
      for (int j = 4 * h; j < 4 * h + 4; ++j) v[j] = copysignf(v[j], y[j]);  // the remainder step turns -0 into +0
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
      p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], p, true);
      w[h] = (uint32_t)p;
    } else {
      // 1.5 * 2^23 + v is rounded to the nearest integer, ties to even, and
      // holds it in its low byte
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = __float_as_uint(v[4 * h + j] + 0x1.8p+23f);
      w[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[3], u[2], 0x0C0C0400u),
                                   __builtin_amdgcn_perm(u[1], u[0], 0x0C0C0400u), 0x05040100u);
    }
  }
  return w[0] | ((uint64_t)w[1] << 32);
}

// WAVES waves hold one row, NCH pieces a thread.  LANES < 64 (one wave): a
// row takes that many lanes, a wave several rows.  One-wave rows share
// workgroups of 256 threads and have no barrier.  WHOLE: the row's length is a
// multiple of 8, so every piece is whole or absent.
template <int LANES, int WAVES, int NCH, bool WHOLE>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void rmsnorm_kernel(coli_moe_rmsnorm_t a) {
  static_assert(LANES == 64 || WAVES == 1, "part of a wave");
  constexpr int kThreads = LANES * WAVES;  // of a row
  __shared__ double sum_of[WAVES];
  __shared__ float max_of[WAVES];
  const int wave = WAVES == 1 ? 0 : (int)(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int tid = WAVES == 1 ? lane % LANES : (int)threadIdx.x;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  int64_t row = block;
  if constexpr (WAVES == 1) {
    row = block * (256 / LANES) + threadIdx.x / LANES;
    if constexpr (LANES == 64) row = uniform((int)row);
    // whole waves without a row leave; in a wave with some, the lanes of the
    // missing rows repeat the last row, with the same results
    const int64_t wave_row = block * (256 / LANES) + (threadIdx.x & ~63) / LANES;
    if (wave_row >= a.rows) return;
    row = row < a.rows ? row : a.rows - 1;
  } else if (row >= a.rows) {
    return;
  }
  const int h = a.hidden;

  // every load is issued before the first value is used
  auto load = [&](const void *base, int type, int64_t first, int c, Raw8 &r) {
    if (!WHOLE)
      r = load_raw8(base, type, first + c, h - c);
    else if (c < h)
      r = load_raw8(base, type, first + c);
  };
  Raw8 xr[NCH], rr[NCH], wr[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = kVec * (i * kThreads + tid);
    load(a.x, a.x_type, row * a.x_stride, c, xr[i]);
    if (a.residual) load(a.residual, a.residual_type, row * a.residual_stride, c, rr[i]);
    if (a.weight) load(a.weight, a.weight_type, 0, c, wr[i]);
  }
  float s[NCH][kVec];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    unpack8(a.x_type, xr[i], s[i]);
    if (a.residual) {
      float r[kVec];
      unpack8(a.residual_type, rr[i], r);
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[i][j] += r[j];
      round8(a.residual_type, s[i]);
    }
    if (WHOLE && kVec * (i * kThreads + tid) >= h)
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[i][j] = 0.0f;
  }
  auto store = [&](void *base, int type, int64_t first, int c, const float (&v)[kVec]) {
    if (!WHOLE)
      store8(base, type, first + c, h - c, v);
    else if (c < h)
      store8(base, type, first + c, v);
  };
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = kVec * (i * kThreads + tid);
      store(a.residual_out, a.residual_type, row * a.residual_out_stride, c, s[i]);
    }
  }

  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) sum = __builtin_fma((double)s[i][j], (double)s[i][j], sum);
  sum = lanes_sum64<LANES>(sum);
  if constexpr (WAVES > 1) {
    if (lane == 0) sum_of[wave] = sum;
    block_barrier();  // for LDS alone: the stores above go on
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) sum += sum_of[i];
  }
  const double mean = sum / (double)h + (double)a.eps;
  // a row of zeros without eps: zeros; of Inf or NaN: NaN (for Inf, by the Newton steps)
  const double r64 = mean != 0.0 ? rsqrt64(mean) : 0.0;
  float r = (float)r64;
  // 1 / rms of a row near either end of float32's range passes the other end,
  // or is subnormal: a power of two goes from r to s, which is exact (elements
  // of s that it makes subnormal give results far below that)
  constexpr int kNormal = 0x108;
  if (!__builtin_amdgcn_classf(r, kNormal)) {
    const float up = r64 > 1.0 ? 0x1p+64f : 0x1p-64f;
    r = (float)(r64 > 1.0 ? r64 * 0x1p-64 : r64 * 0x1p+64);
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[i][j] *= up;
  }
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) s[i][j] *= r;
    if (a.weight) {
      float w[kVec];
      unpack8(a.weight_type, wr[i], w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[i][j] *= w[j];
    }
  }

  if (a.out_type <= COLI_MOE_F16) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = kVec * (i * kThreads + tid);
      store(a.out, a.out_type, row * a.out_stride, c, s[i]);
    }
    return;
  }

  // 8 bits: the largest magnitude of the row or of each group (pieces past
  // the row's end hold zeros), then the codes
  const bool e4m3 = a.out_type == COLI_MOE_E4M3, finite = r == r;  // the maxima leave NaNs out
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
    all = lanes_max<LANES>(all);
    if constexpr (WAVES > 1) {
      if (lane == 0) max_of[wave] = all;
      block_barrier();
#pragma unroll
      for (int i = 0; i < WAVES; ++i) all = fmaxf(all, max_of[i]);
    }
    const float scale = finite ? all / q : r;
    if (tid == 0) a.scales[row * a.scales_stride] = scale;
#pragma unroll
    for (int i = 0; i < NCH; ++i) m[i] = scale;
  } else {
    // a group's pieces sit in 8 or 16 neighbouring lanes
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      m[i] = (a.group == 64 ? lanes_max<8>(m[i]) : lanes_max<16>(m[i])) / q;
      if (!finite) m[i] = r;
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
    if (WHOLE || h - c >= kVec)
      __builtin_memcpy(out, &codes, 8);
    else
      for (int j = 0; j < h - c; ++j) out[j] = (uint8_t)(codes >> (8 * j));
  }
}

template <int LANES, int WAVES, int NCH>
hipError_t launch_shape(const coli_moe_rmsnorm_t &a, hipStream_t s) {
  constexpr int kRows = WAVES == 1 ? 256 / LANES : 1;
  // threads along one axis of a grid are counted in 32 bits
  constexpr uint32_t kMaxX = 1u << 20;
  const uint32_t blocks = (uint32_t)(((int64_t)a.rows + kRows - 1) / kRows);
  const dim3 grid(blocks < kMaxX ? blocks : kMaxX, (blocks + kMaxX - 1) / kMaxX), block(WAVES == 1 ? 256 : 64 * WAVES);
  return a.hidden % kVec == 0 ? launch(rmsnorm_kernel<LANES, WAVES, NCH, true>, grid, block, 0, s, a)
                              : launch(rmsnorm_kernel<LANES, WAVES, NCH, false>, grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_rmsnorm(const coli_moe_rmsnorm_t &a, hipStream_t s) {
  const int pieces = (a.hidden + kVec - 1) / kVec;
  // one piece a thread: fewer threads with more pieces each are slower where
  // there are few rows (6144 columns, one row: 12 waves 3.2 us, 8 of two
  // pieces 4.6, 4 of three 4.8).  Except many rows of 12 waves: a CU holds two
  // such workgroups, 24 of its 32 waves, but four of 8 waves with two pieces
  // (6144 columns of bf16: 512 rows 10.6 us against 10.8, 4096 rows 45.4
  // against 41.7).
  if (pieces <= 16) return launch_shape<16, 1, 1>(a, s);
  if (pieces <= 64) return launch_shape<64, 1, 1>(a, s);
  if (pieces <= 128) return launch_shape<64, 2, 1>(a, s);
  if (pieces <= 256) return launch_shape<64, 4, 1>(a, s);
  if (pieces <= 384) return launch_shape<64, 6, 1>(a, s);
  if (pieces <= 512) return launch_shape<64, 8, 1>(a, s);
  if (pieces <= 768) return a.rows <= 1024 ? launch_shape<64, 12, 1>(a, s) : launch_shape<64, 8, 2>(a, s);
  if (pieces <= 1024) return launch_shape<64, 16, 1>(a, s);
  if (pieces <= 2048) return launch_shape<64, 16, 2>(a, s);
  return launch_shape<64, 16, 4>(a, s);
}

}  // namespace coli
