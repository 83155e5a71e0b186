// Rotary positions (coli_moe_rotary): pairs of a head turned by
// position * frequency.
//
// Bound by bytes (each element read and written once); the angles are shared
// by all heads of a token, so a workgroup takes whole tokens, computes their
// cosines and sines into LDS once and turns every head with them.  4096 tokens
// of 56 heads of 128 halves, 64 of them turned: 24 us for 117 MB (4.9 TB/s; a
// large copy 5.1).  Results of 1024 tokens and more are stored past the caches:
// with them, 37 us back to back (what a kernel that reads the result next makes
// of it was not measured).  One token of 72 heads: 3 us, a launch.
#include "element_types.h"
#include "internal.h"
#include "kv_cache.h"

namespace coli {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kMaxPairs = 2048;  // part / 2 at most

// cos and sin of p * f.  The product is a float64 with the rest that it was
// rounded by, and 1 / (2 pi) has two parts, so that for |p| < 2^53 the turns are
// off by less than 2^-50 when they are reduced to [-1/2, 1/2]; what float32 sees
// is an angle in [-1, 1] half turns with its own rounding.  (One product by one
// part was off by 2^-27 turns at positions of 2^28, by all of one at 2^53.)
__device__ __forceinline__ float2 turn(double p, float f, float scale, bool inverse) {
  constexpr double kInv = 0x1.45f306dc9c883p-3, kInvRest = -0x1.6b01ec5417056p-57;
  const double angle = p * (double)f, rest = __builtin_fma(p, (double)f, -angle), turns = angle * kInv;
  double part = __builtin_fma(angle, kInvRest, __builtin_fma(rest, kInv, __builtin_fma(angle, kInv, -turns)));
  part += turns - rint(turns);
  part -= rint(part);
  float c, s;
  sincospif(2.0f * (float)part, &s, &c);
  return make_float2(scale * c, inverse ? -scale * s : scale * s);
}

struct RotaryShape {
  int pair_units, copy_units;  // pieces of a head: turned (8 pairs, or 8 elements interleaved) and copied
  int units;                   // of all heads of a token
};

// Eight waves a SIMD: more than 96 scalar registers cost the prompt above 1.4 us.
template <bool kPast>
__global__ __launch_bounds__(kRotaryThreads, 8) void rotary_kernel(coli_moe_rotary_t a, RotaryShape sh, int split) {
  __shared__ float2 cs[kMaxPairs];
  const int half = a.part / 2;
  auto store = [&](int64_t i, int n, const float (&v)[8]) {
    if constexpr (kPast)
      store8_past(a.out, a.type, i, n, v);
    else
      store8(a.out, a.type, i, n, v);
  };
  // split: consecutive workgroups that share a token's units
  for (int64_t w = blockIdx.x; w < (int64_t)a.tokens * split; w += gridDim.x) {
    const int64_t t = w / split;
    const int part = (int)(w % split);
    const double p = a.wide ? (double)static_cast<const int64_t *>(a.positions)[t]
                            : (double)static_cast<const int32_t *>(a.positions)[t];
    __syncthreads();
    for (int i = threadIdx.x; i < half; i += kRotaryThreads) cs[i] = turn(p, a.freq[i], a.scale, a.inverse);
    __syncthreads();
    const int per_head = sh.pair_units + sh.copy_units;
    for (int u = part * kRotaryThreads + threadIdx.x; u < sh.units; u += split * kRotaryThreads) {
      const int head = u / per_head, k = u % per_head;
      const int64_t x = t * a.x_token + head * a.x_head, o = t * a.out_token + head * a.out_head;
      float v[8], y[8];
      if (k >= sh.pair_units) {
        const int c = a.part + 8 * (k - sh.pair_units), n = a.dim - c;
        unpack8(a.type, load_raw8(a.x, a.type, x + c, n), v);
        store(o + c, n, v);
      } else if (a.interleaved) {
        const int c = 8 * k, n = a.part - c;
        unpack8(a.type, load_raw8(a.x, a.type, x + c, n), v);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 e = cs[min((c + j) / 2, half - 1)];
          y[j] = __builtin_fmaf(v[j], e.x, -(v[j + 1] * e.y));
          y[j + 1] = __builtin_fmaf(v[j], e.y, v[j + 1] * e.x);
        }
        store(o + c, n, y);
      } else {
        const int c = 8 * k, n = half - c;
        float b[8], z[8];
        const Raw8 r0 = load_raw8(a.x, a.type, x + c, n), r1 = load_raw8(a.x, a.type, x + half + c, n);
        unpack8(a.type, r0, v);
        unpack8(a.type, r1, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 e = cs[min(c + j, half - 1)];
          y[j] = __builtin_fmaf(v[j], e.x, -(b[j] * e.y));
          z[j] = __builtin_fmaf(v[j], e.y, b[j] * e.x);
        }
        store(o + c, n, y);
        store(o + half + c, n, z);
      }
    }
  }
}

}  // namespace

hipError_t launch_rotary(const coli_moe_rotary_t &a, hipStream_t s) {
  RotaryShape sh;
  const int half = a.part / 2;
  sh.pair_units = a.interleaved ? (a.part + 7) / 8 : (half + 7) / 8;
  // in place, what is not turned stays where it is
  sh.copy_units = a.out == a.x ? 0 : (a.dim - a.part + 7) / 8;
  sh.units = a.heads * (sh.pair_units + sh.copy_units);
  if (sh.units == 0) return hipSuccess;
  const int blocks = (sh.units + kRotaryThreads - 1) / kRotaryThreads;
  const int split = a.tokens >= 1024 ? 1 : blocks < 8 ? blocks : 8;
  const int64_t work = (int64_t)a.tokens * split;
  return launch(split == 1 ? rotary_kernel<true> : rotary_kernel<false>,
                dim3((unsigned)(work < (1 << 20) ? work : 1 << 20)), dim3(kRotaryThreads), 0, s, a, sh, split);
}

}  // namespace coli
