// The paged 4-bit key/value cache: append (quantise), read (expand) and
// eviction by accumulated attention weight.  The attention over it is in
// attention.hip.
#include "element_types.h"
#include "internal.h"
#include "kv_cache.h"
#include "wave.h"

namespace coli {
namespace {

constexpr int kRowThreads = 256;

// Code of x for the scale s (> 0, finite): x / s rounded to the nearest, ties
// to even, held within [-7, 7].  x and s are 24- and 8-bit numbers, so the
// quotient's rounding to float32 could only put it on a border from just
// beside it; the remainder d = x - q s is exact and tells.
__device__ __forceinline__ int code4(float x, float s) {
  const float y = fminf(fmaxf(x / s, -8.0f), 8.0f);
  float q = rintf(y);
  const float d = __builtin_fmaf(-q, s, x), h = 0.5f * s;
  if (fabsf(q) < 8.0f) {
    if (d > h || (d == h && ((int)q & 1)))
      q += 1.0f;
    else if (d < -h || (d == -h && ((int)q & 1)))
      q -= 1.0f;
  }
  return (int)fminf(fmaxf(q, -7.0f), 7.0f);
}

// Eight columns a thread, eight threads a scale: a wave takes eight groups of
// one token at a time, of its keys and then its values.
__global__ __launch_bounds__(kRowThreads) void kv_append_kernel(KvView kv, coli_moe_kv_rows_t r,
                                                                coli_moe_kv_values_t a, int parts) {
  const int lane = threadIdx.x & 63, D = kv.p.head_dim, ng = D / kKvGroup;
  const int groups = 2 * kv.p.kv_heads * ng;
  const int64_t waves = (int64_t)gridDim.x * (kRowThreads / 64);
  for (int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + uniform(threadIdx.x >> 6);
       w < (int64_t)r.tokens * parts; w += waves) {
    const int t = (int)(w / parts), part = (int)(w % parts);
    const int s = find_seq(r, t);
    if (s < 0) continue;
    const int64_t row = token_row(r, s, t);
    const int page = row_page(kv, r.table + s * r.table_stride, r.table_width, row);
    if (page < 0) continue;
    const int slot = (int)row & (kv.p.page_size - 1);
    for (int g0 = part * 8; g0 < groups; g0 += parts * 8) {
      const int gi = g0 + lane / 8;
      const bool live = gi < groups;  // all lanes take part in the maximum
      const bool is_v = gi >= groups / 2;
      const int hg = is_v ? gi - groups / 2 : gi, h = hg / ng, g = hg % ng;
      const int col = g * kKvGroup + (lane & 7) * 8;
      float x[8];
      if (live)
        unpack8(a.type, is_v ? load_raw8(a.v, a.type, t * a.v_token + h * a.v_head + col)
                             : load_raw8(a.k, a.type, t * a.k_token + h * a.k_head + col), x);
      else
        for (int j = 0; j < 8; ++j) x[j] = 0.0f;
      // as integers: Inf and NaN are above every finite value
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
      top = max(top, (uint32_t)__shfl_xor((int)top, 1));
      top = max(top, (uint32_t)__shfl_xor((int)top, 2));
      top = max(top, (uint32_t)__shfl_xor((int)top, 4));
      if (!live) continue;
      // the quotient in float32 never falls on a bfloat16 border that the exact one is not on
      const uint16_t sb = top >= 0x7F800000u ? 0x7FC0 : to_bf16(__uint_as_float(top) / 7.0f);
      const float sc = from_bf16(sb);
      uint32_t codes = 0;
      if (sc > 0.0f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) codes |= (uint32_t)(code4(x[j], sc) & 15) << (4 * j);
      }
      const int64_t ph = (int64_t)page * kv.p.kv_heads + h;
      uint8_t *cp = (is_v ? kv.p.v_codes : kv.p.k_codes) + (ph * kv.p.page_size + slot) * (D / 2) + col / 2;
      *reinterpret_cast<uint32_t *>(cp) = codes;
      if ((lane & 7) == 0) {
        (is_v ? kv.p.v_scales : kv.p.k_scales)[(ph * ng + g) * kv.p.page_size + slot] = sb;
        if (kv.p.weights && g == 0 && !is_v) kv.p.weights[ph * kv.p.page_size + slot] = 0.0f;
      }
    }
  }
}

// Eight columns a thread; a wave takes 512 columns of one token at a time.
__global__ __launch_bounds__(kRowThreads) void kv_read_kernel(KvView kv, coli_moe_kv_rows_t r, coli_moe_kv_values_t a,
                                                              int parts) {
  const int lane = threadIdx.x & 63, D = kv.p.head_dim, ng = D / kKvGroup;
  const int units = 2 * kv.p.kv_heads * (D / 8);
  const int64_t waves = (int64_t)gridDim.x * (kRowThreads / 64);
  for (int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + uniform(threadIdx.x >> 6);
       w < (int64_t)r.tokens * parts; w += waves) {
    const int t = (int)(w / parts), part = (int)(w % parts);
    const int s = find_seq(r, t);
    if (s < 0) continue;
    const int64_t row = token_row(r, s, t);
    const int page = row_page(kv, r.table + s * r.table_stride, r.table_width, row);
    const int slot = (int)row & (kv.p.page_size - 1);
    for (int u = part * 64 + lane; u < units; u += parts * 64) {
      const bool is_v = u >= units / 2;
      const int hu = is_v ? u - units / 2 : u, h = hu / (D / 8), col = hu % (D / 8) * 8;
      float x[8] = {};
      if (page >= 0) {
        const int64_t ph = (int64_t)page * kv.p.kv_heads + h;
        const uint8_t *cp = (is_v ? kv.p.v_codes : kv.p.k_codes) + (ph * kv.p.page_size + slot) * (D / 2) + col / 2;
        const int c = *reinterpret_cast<const int *>(cp);
        const float sc = from_bf16(
            (is_v ? kv.p.v_scales : kv.p.k_scales)[(ph * ng + col / kKvGroup) * kv.p.page_size + slot]);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (float)((c << (28 - 4 * j)) >> 28) * sc;
      }
      if (is_v)
        store8(a.v, a.type, t * a.v_token + h * a.v_head + col, x);
      else
        store8(a.k, a.type, t * a.k_token + h * a.k_head + col, x);
    }
  }
}

// ---------------------------------------------------------------------------
// Eviction
// ---------------------------------------------------------------------------

constexpr int kSelectThreads = 1024;

// Weights in an order of unsigned integers: larger weights larger, NaN above
// everything, -0 as 0.
__device__ __forceinline__ uint32_t rank_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t row_key(const KvView &kv, const int32_t *table, int width, int h, int row) {
  const int page = row_page(kv, table, width, row);
  if (page < 0) return rank_key(0.0f);
  return rank_key(kv.p.weights[(((int64_t)page * kv.p.kv_heads + h) << kv.shift) + (row & (kv.p.page_size - 1))]);
}

// Sum of v over the threads before this one, and over all (*total).
__device__ __forceinline__ int block_scan(int v, int *lds, int *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kSelectThreads / 64; ++i) {
    if (i < wave) before += lds[i];
    all += lds[i];
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

// The rows that one sequence's key head keeps: the c-th largest key of the
// middle rows is found digit by digit (8 bits, largest first), then rows in
// order are kept while they are first, recent, above it, or among the first
// of those equal to it.
__global__ __launch_bounds__(kSelectThreads) void kv_select_kernel(KvView kv, coli_moe_kv_rows_t r,
                                                                   coli_moe_kv_evict_t a) {
  __shared__ int hist[256];
  __shared__ int scan[kSelectThreads / 64];
  __shared__ int chosen[2];  // digit, rows still to take below it
  const int H = kv.p.kv_heads, tid = threadIdx.x;
  for (int64_t w = blockIdx.x; w < (int64_t)r.seqs * H; w += gridDim.x) {
    const int s = (int)(w / H), h = (int)(w % H);
    const int32_t *table = r.table + s * r.table_stride;
    // lengths may be anything; at most 2^30 rows stand in a table
    const int len = min(max(r.lengths[s], 0), r.table_width << kv.shift);
    const int keep = min(a.keep, len);
    int32_t *kept = a.kept + w * a.keep;
    if (h == 0 && tid == 0) a.new_lengths[s] = keep;
    for (int i = keep + tid; i < a.keep; i += kSelectThreads) kept[i] = -1;
    if (len <= a.keep) {
      for (int i = tid; i < keep; i += kSelectThreads) kept[i] = i;
      continue;
    }
    const int lo = a.first, hi = len - a.recent;
    int need = keep - a.first - a.recent;  // of the middle rows, 0 .. hi - lo
    uint32_t key = 0, known = 0;           // digits found so far, and their mask
    if (need > 0) {
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        for (int row = lo + tid; row < hi; row += kSelectThreads) {
          const uint32_t k = row_key(kv, table, r.table_width, h, row);
          if ((k & known) == key) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        // rows in digits above d, from the largest digit down
        const int v = tid < 256 ? hist[255 - tid] : 0;
        int total;
        const int before = block_scan(v, scan, &total);
        if (tid < 256 && before < need && before + v >= need) {
          chosen[0] = 255 - tid;
          chosen[1] = need - before;
        }
        __syncthreads();
        key |= (uint32_t)chosen[0] << shift;
        known |= 255u << shift;
        need = chosen[1];
        __syncthreads();
      }
    }
    // need: rows equal to `key` still to take, in order (0 when no middle row is kept)
    const bool any = keep > a.first + a.recent;
    int out = 0, equal = 0;
    for (int base = 0; base < len; base += kSelectThreads) {
      const int row = base + tid;
      const bool middle = row >= lo && row < hi;
      const uint32_t k = middle && any ? row_key(kv, table, r.table_width, h, row) : 0;
      const int same = middle && any && k == key ? 1 : 0;
      int sames, takes;
      const int rank = equal + block_scan(same, scan, &sames);
      const int take = row < len && (!middle || (any && (k > key || (same && rank < need)))) ? 1 : 0;
      const int at = out + block_scan(take, scan, &takes);
      if (take) kept[at] = row;
      equal += sames;
      out += takes;
    }
  }
}

// Copies the kept rows: 16 bytes a thread, rows of one head side by side.
__global__ __launch_bounds__(kRowThreads) void kv_move_kernel(KvView kv, coli_moe_kv_rows_t r, coli_moe_kv_evict_t a,
                                                              int chunks) {
  const int H = kv.p.kv_heads, D = kv.p.head_dim, ng = D / kKvGroup, ps = kv.p.page_size;
  const int pieces = D / 32;  // 16-byte pieces of a row of codes
  const int rows = kRowThreads / pieces;
  for (int64_t w = blockIdx.x; w < (int64_t)r.seqs * H * chunks; w += gridDim.x) {
    const int64_t sh = w / chunks;
    const int s = (int)(sh / H), h = (int)(sh % H);
    const int i = (int)(w % chunks) * rows + threadIdx.x / pieces, piece = threadIdx.x % pieces;
    if (i >= a.keep) continue;
    const int row = a.kept[sh * a.keep + i];
    if (row < 0) continue;
    const int from = row_page(kv, r.table + s * r.table_stride, r.table_width, row);
    const int to = row_page(kv, a.into + s * a.into_stride, a.into_width, i);
    if (from < 0 || to < 0) continue;
    const int64_t src = (int64_t)from * H + h, dst = (int64_t)to * H + h;
    const int ss = row & (ps - 1), ds = i & (ps - 1);
    const int64_t sb = (src * ps + ss) * (D / 2) + piece * 16, db = (dst * ps + ds) * (D / 2) + piece * 16;
    const uint4 k = *reinterpret_cast<const uint4 *>(kv.p.k_codes + sb);
    const uint4 v = *reinterpret_cast<const uint4 *>(kv.p.v_codes + sb);
    *reinterpret_cast<uint4 *>(kv.p.k_codes + db) = k;
    *reinterpret_cast<uint4 *>(kv.p.v_codes + db) = v;
    if (piece < ng) {
      const int64_t si = (src * ng + piece) * ps + ss, di = (dst * ng + piece) * ps + ds;
      kv.p.k_scales[di] = kv.p.k_scales[si];
      kv.p.v_scales[di] = kv.p.v_scales[si];
    }
    if (piece == 0) kv.p.weights[dst * ps + ds] = kv.p.weights[src * ps + ss];
  }
}

unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20); }

}  // namespace

hipError_t launch_kv_append(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_values_t &a,
                            hipStream_t s) {
  const int groups = 2 * kv.kv_heads * (kv.head_dim / kKvGroup), steps = (groups + 7) / 8;
  const int parts = r.tokens >= 2048 ? 1 : steps;  // few tokens: a wave per eight groups
  const int64_t blocks = ((int64_t)r.tokens * parts + kRowThreads / 64 - 1) / (kRowThreads / 64);
  return launch(kv_append_kernel, dim3(grid_of(blocks)), dim3(kRowThreads), 0, s, kv_view(kv), r, a, parts);
}

hipError_t launch_kv_read(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_values_t &a,
                          hipStream_t s) {
  const int units = 2 * kv.kv_heads * (kv.head_dim / 8), steps = (units + 63) / 64;
  const int parts = r.tokens >= 2048 ? 1 : steps;
  const int64_t blocks = ((int64_t)r.tokens * parts + kRowThreads / 64 - 1) / (kRowThreads / 64);
  return launch(kv_read_kernel, dim3(grid_of(blocks)), dim3(kRowThreads), 0, s, kv_view(kv), r, a, parts);
}

hipError_t launch_kv_evict(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_evict_t &a,
                           hipStream_t s) {
  const int64_t heads = (int64_t)r.seqs * kv.kv_heads;
  const hipError_t e = launch(kv_select_kernel, dim3(grid_of(heads)), dim3(kSelectThreads), 0, s, kv_view(kv), r, a);
  if (e != hipSuccess) return e;
  const int rows = kRowThreads / (kv.head_dim / 32), chunks = (a.keep + rows - 1) / rows;
  return launch(kv_move_kernel, dim3(grid_of(heads * chunks)), dim3(kRowThreads), 0, s, kv_view(kv), r, a, chunks);
}

}  // namespace coli
