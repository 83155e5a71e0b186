// What the kernels of attention over the 4-bit cache share: the call, codes
// as halves, and where keys stand.
#pragma once

#include "element_types.h"
#include "internal.h"
#include "kv_cache.h"
#include "wave.h"

namespace coli {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));

constexpr int kTileThreads = 256;
constexpr int kTileWaves = kTileThreads / 64;
constexpr float kLog2e = 1.44269504088896340736f;

// A weight is exp2((u x - m) cs) with the power of two u and the maximum m of
// u x.  One multiply-add, x (u cs) - m cs, has the rounding of m cs, common to
// all keys of a row but not to its other maxima; so above this size of m cs the
// difference is taken first.
constexpr float kFar = 16.0f;

// The maximum that a row's sums stand against may be passed by 2^kSlack before
// they are brought to a new one.
constexpr float kSlack = 8.0f;

// A weight exp2((v - m) cs) / sum from a score v computed once more.  Scores too
// large for float32 to tell apart may pass m by far then, so 2^-kSlack of the
// exponential is held within 2^-kSlack of the row's sum: a weight is at most 1.
// share_again takes both back.  A NaN row's share is NaN.
__device__ __forceinline__ float weight_again(float difference, float cs, float limit) {
  return __builtin_amdgcn_fmed3f(__builtin_amdgcn_exp2f(__builtin_fmaf(difference, cs, -kSlack)), 0.0f, limit);
}
__device__ __forceinline__ float limit_again(float sum) { return sum * 0x1p-8f; }
__device__ __forceinline__ float share_again(float sum) { return sum != 0.0f ? 0x1p8f / sum : 0.0f; }

// Adds to a place of weights_out, which several sequences may share: each adds
// its own sum, once, in no order.
__device__ __forceinline__ void add_weight(float *to, float v) { unsafeAtomicAdd(to, v); }

// Power of two that brings v (>= 0) into [2^14, 2^15), within float32's range,
// and its inverse.
__device__ __forceinline__ int lift_exponent(float v) { return max((int)(__float_as_uint(v) >> 23) & 255, 20); }
__device__ __forceinline__ float lift(int ex) { return __uint_as_float((uint32_t)(268 - ex) << 23); }
__device__ __forceinline__ float unlift(int ex) { return __uint_as_float((uint32_t)(ex - 14) << 23); }

// The signed codes at bits 0 and 16 (4 and 20) of w: the exclusive or with 8
// that makes u of a code and the exponent of 1024 are one constant, so the two
// masks are one three-input instruction.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {
  const half2_t v = __builtin_bit_cast(half2_t, (w & 0x000F000Fu) ^ 0x64086408u);
  return __builtin_bit_cast(uint32_t, v + half2_t{(_Float16)-1032.0f, (_Float16)-1032.0f});
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) {
  const half2_t v = __builtin_bit_cast(half2_t, (w & 0x00F000F0u) ^ 0x64806480u);
  const half2_t by = {(_Float16)0.0625f, (_Float16)0.0625f}, off = {(_Float16)-72.0f, (_Float16)-72.0f};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v, by, off));
}

// The 8 codes of a dword as halves, in the order (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ half8_t codes_of(uint32_t w) {
  u32x4 r;
  r[0] = low_codes(w);
  r[1] = high_codes(w);
  w >>= 8;
  r[2] = low_codes(w);
  r[3] = high_codes(w);
  return __builtin_bit_cast(half8_t, r);
}

struct Call {
  KvView kv;
  coli_moe_kv_rows_t rows;
  coli_moe_kv_attention_t a;
  float cs;        // a score q . k times this is a power of two's exponent: |scale| log2 e (the sign goes with q)
  int group;       // query heads of a key head
  int tiles;       // tiles of a sequence's key head that the grid has
  int tile_waves;  // of them in one workgroup (1, 2 or 4)
  int few_rows;    // a key head's query rows up to which a sequence takes the tiles of 16 columns
  int waves;       // of a workgroup of tiles, 4 or 8
  int splits, prompt_splits;  // of the keys, by the tiles and by the prompts' kernel
  int part_splits;  // the larger
  float *part_o;   // [row][split][D], row = token * q_heads + head
  float2 *part_ml; // [row][split] maximum (of scores without cs) and sum
  float2 *ml;      // [row], for the weights; NULL: not wanted
  char *q_halves;  // for the weights of more rows than a tile: [key head][token][head of the group][D] halves
  float4 *q_info;  // and each row's power of two, its maximum, share_again and limit_again
  int blocks;      // workgroups of the tiles' kernel that take tiles; those after them copy weights
  int copy_parts;  // of a sequence's key head, whose weights go to weights_out before the sums do; 0: they are there
};

// Range of keys that the rows r0 .. r1 of a sequence's key head see.
struct KeyRange {
  int64_t lo, hi;
};
__device__ __forceinline__ KeyRange keys_of_rows(const Call &c, SeqSpan span, int64_t len, int r0, int r1) {
  const int64_t p0 = len - span.n + r0 / c.group, p1 = len - span.n + r1 / c.group;
  const int64_t cap = (int64_t)c.rows.table_width << c.kv.shift;
  KeyRange k;
  k.hi = min(p1 + 1, cap);
  k.lo = c.a.window ? max(p0 - c.a.window + 1, (int64_t)0) : 0;
  return k;
}

// Rows of a workgroup of the prompts' kernel.  D = 256 has four waves of twice
// the registers: the results of 32 rows alone fill half of 256.
constexpr int prompt_rows(int dim) { return dim == 256 ? 128 : 256; }
hipError_t launch_attention_prompts(const Call &c, hipStream_t s);
hipError_t launch_row_weights(const Call &c, hipStream_t s);

// Where a step's two 16 keys stand: uniform.  Pages of 16 rows: two places, else
// one after the other.  The table's entries are asked for a step before they
// are needed, as they stand.
template <bool kSmallPages>
struct Entries {
  int entry[kSmallPages ? 2 : 1];
};
template <bool kSmallPages>
struct Place {
  uint64_t row[kSmallPages ? 2 : 1];    // of codes
  uint64_t scale[kSmallPages ? 2 : 1];  // first scale of group 0
  bool ok[2];
};

template <bool kSmallPages>
__device__ __forceinline__ Entries<kSmallPages> entries_of(const Call &c, const int32_t *table, int key0) {
  Entries<kSmallPages> e;
#pragma unroll
  for (int t = 0; t < (kSmallPages ? 2 : 1); ++t)
    e.entry[t] = table[min((key0 >> c.kv.shift) + t, c.rows.table_width - 1)];
  return e;
}

template <int D, bool kSmallPages>
__device__ __forceinline__ Place<kSmallPages> place_of(const Call &c, const Entries<kSmallPages> &e, int h, int key0) {
  Place<kSmallPages> p;
  const int slot = kSmallPages ? 0 : key0 & (c.kv.p.page_size - 1);
#pragma unroll
  for (int t = 0; t < (kSmallPages ? 2 : 1); ++t) {
    const int entry = uniform(e.entry[t]);
    p.ok[t] = (key0 >> c.kv.shift) + t < c.rows.table_width && (unsigned)entry < (unsigned)c.kv.p.n_pages;
    const int page = p.ok[t] ? entry : 0;
    p.row[t] = code_row(c.kv, page, h, slot);
    p.scale[t] = scale_index<D / kKvGroup>(c.kv, page, h, 0, slot);
  }
  if constexpr (!kSmallPages) p.ok[1] = p.ok[0];
  return p;
}

}  // namespace coli
