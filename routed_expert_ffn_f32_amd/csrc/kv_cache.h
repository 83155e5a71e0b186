// The paged 4-bit key/value cache (coli_moe_kv_t) as kernels see it: where a
// row stands, which sequence a token belongs to, and the limits that
// attention.hip, kv_cache.hip and operators.hip share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "coli_moe.h"
#include "internal.h"
#include "wave.h"

namespace coli {

constexpr int kKvGroup = 64;  // columns of one scale

struct KvView {
  coli_moe_kv_t p;
  int shift;  // log2(page_size)
};

inline KvView kv_view(const coli_moe_kv_t &kv) { return {kv, __builtin_ctz((unsigned)kv.page_size)}; }

// First token and number of tokens of sequence s.
struct SeqSpan {
  int first, n;
};

__device__ __forceinline__ SeqSpan seq_span(const coli_moe_kv_rows_t &r, int s) {
  if (!r.offsets) return {s, 1};
  const int a = min(max(r.offsets[s], 0), r.tokens), b = min(max(r.offsets[s + 1], 0), r.tokens);
  return {a, max(b - a, 0)};
}

// The sequence of token t, -1 for none: called by whole waves with one t.
// Each step splits the range in 64 and counts the bounds at or below t.
__device__ __forceinline__ int find_seq(const coli_moe_kv_rows_t &r, int t) {
  if (!r.offsets) return t;
  const int lane = threadIdx.x & 63;
  int lo = 0, n = r.seqs;
  while (n > 1) {
    const int step = (n + 63) / 64, i = lane * step;
    const bool below = i < n && r.offsets[lo + i] <= t;
    const int k = __popcll(__ballot(below));
    if (k == 0) return -1;
    lo += (k - 1) * step;
    n = min(step, n - (k - 1) * step);
  }
  lo = uniform(lo);
  return r.offsets[lo] <= t && t < r.offsets[lo + 1] ? lo : -1;
}

// Page of rows row .. of sequence s, -1 where none is.
__device__ __forceinline__ int row_page(const KvView &kv, const int32_t *table, int width, int64_t row) {
  const int64_t i = row >> kv.shift;
  if (i < 0 || i >= width) return -1;
  const int page = table[i];
  return (unsigned)page < (unsigned)kv.p.n_pages ? page : -1;
}

// Index of a row of codes, and of the scale of its group g (kv.weights: that of
// a row).  One 64-bit multiplication each: a page's rows of all heads are fewer
// than 2^21 scales.
__device__ __forceinline__ uint64_t code_row(const KvView &kv, int page, int h, int slot) {
  return (uint64_t)(uint32_t)page * (uint32_t)(kv.p.kv_heads << kv.shift) + (uint32_t)((h << kv.shift) + slot);
}
template <int kGroups>
__device__ __forceinline__ uint64_t scale_index(const KvView &kv, int page, int h, int g, int slot) {
  return (uint64_t)(uint32_t)page * (uint32_t)((kv.p.kv_heads * kGroups) << kv.shift) +
         (uint32_t)(((h * kGroups + g) << kv.shift) + slot);
}

hipError_t launch_rotary(const coli_moe_rotary_t &a, hipStream_t s);  // tokens >= 1
hipError_t launch_kv_append(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_values_t &a,
                            hipStream_t s);  // tokens >= 1, as below
hipError_t launch_kv_read(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_values_t &a,
                          hipStream_t s);
hipError_t launch_kv_evict(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_evict_t &a,
                           hipStream_t s);
size_t kv_attention_workspace_bytes(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r,
                                    const coli_moe_kv_attention_t &a);
hipError_t launch_kv_attention(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_attention_t &a,
                               void *workspace, hipStream_t s);

}  // namespace coli
