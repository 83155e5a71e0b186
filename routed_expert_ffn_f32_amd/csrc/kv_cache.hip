// The paged 4-bit key/value cache: append (quantise), read (expand) and
// eviction by accumulated attention weight.  The attention over it is in
// attention.hip.
//
// Few tokens are bound by the loads that follow each other (sequence, length,
// page, rows), so eight tokens' places are looked up together, and there are as
// many waves as one round of them can be: 64 tokens, 8 heads of 128: 5 us to
// append, 4 to read.  Many tokens: read is bound by bytes, append by its
// instructions.  4889 tokens, 4 heads of 256 halves: 16 us to append (25 MB, 5 us
// at a copy's rate; a wave's eight groups of 64 columns are 330 vector
// instructions, 10.6 us of issue in all), 12 to read as float32 (45 MB).  61575
// rows of 8 heads of 128 read as halves, 319 MB: 87 us (3.7 TB/s); reads of many
// tokens are stored past the caches (with them, an eviction and this read take 166
// us back to back instead of 147; what a kernel that reads the result next makes
// of it was not measured).
#include "element_types.h"
#include "internal.h"
#include "kv_cache.h"
#include "wave.h"

namespace coli {
namespace {

constexpr int kRowThreads = 256;

// Code of x for the scale s (> 0, finite; r near 1 / s): x / s rounded to the
// nearest, ties to even, held within [-7, 7].  x r may round to the integer
// beside the right one; d = x - q s is exact (s has 8 bits) and tells.
__device__ __forceinline__ int code4(float x, float s, float r) {
  float q = rintf(x * r);
  const float d = __builtin_fmaf(-q, s, x), h = 0.5f * s;
  if (fabsf(d) > h || (fabsf(d) == h && ((int)q & 1))) q += __builtin_copysignf(1.0f, d);
  return (int)fminf(fmaxf(q, -7.0f), 7.0f);
}

// Where up to kGroup consecutive tokens from t0 on stand: lane i < kGroup gets
// token t0 + i's page (-1: none) and slot, and whether a sequence has it.  The
// first token's sequence is searched, the others' are counted from there, so
// that the lookups of all are under way together.
constexpr int kGroup = 8;
struct Located {
  int page, slot;
  bool in_seq;
};

__device__ __forceinline__ Located locate(const KvView &kv, const coli_moe_kv_rows_t &r, int t0) {
  const int lane = threadIdx.x & 63, t = min(t0 + min(lane, kGroup - 1), r.tokens - 1);
  int s = t, first = t, last = t + 1, len = 0;  // the token's sequence, its bounds and length
  if (!r.offsets) {
    len = r.lengths[s];
  } else if (r.seqs < 64) {
    // every bound and length at once, a lane each
    const int bound = r.offsets[min(lane, r.seqs)], lens = r.lengths[min(lane, r.seqs - 1)];
    s = 0;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const int k = __popcll(__ballot(lane < r.seqs && bound <= min(t0 + i, r.tokens - 1)));
      if (lane == i) s = max(k - 1, 0);
    }
    first = __shfl(bound, s);
    last = __shfl(bound, s + 1);
    len = __shfl(lens, s);
  } else {
    // the last sequence that starts at or before t0, 0 for none
    int lo = 0, n = r.seqs;
    while (n > 1) {
      const int step = (n + 63) / 64, i = lane * step;
      const int k = __popcll(__ballot(i < n && r.offsets[lo + i] <= t0));
      lo += max(k - 1, 0) * step;
      n = k == 0 ? 1 : min(step, n - (k - 1) * step);
    }
    lo = uniform(lo);
    const int bound = r.offsets[min(lo + 1 + lane, r.seqs)];
    s = lo;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      // sequences that start at or before the token, among the next 64
      const int k = __popcll(__ballot(lo + 1 + lane < r.seqs && bound <= min(t0 + i, r.tokens - 1)));
      if (lane == i) s = lo + k;
    }
    // more than 64 sequences begin within the group (all but a few are empty): on from there
    if (s == lo + 64)
      while (s + 1 < r.seqs && r.offsets[s + 1] <= t) ++s;
    first = r.offsets[s], last = r.offsets[s + 1], len = r.lengths[s];
  }
  Located l;
  l.in_seq = t0 + lane < r.tokens && lane < kGroup && first <= t && t < last;
  const int64_t row = (int64_t)len - (min(last, r.tokens) - t);
  l.page = l.in_seq ? row_page(kv, r.table + s * r.table_stride, r.table_width, row) : -1;
  l.slot = (int)row & (kv.p.page_size - 1);
  return l;
}

// Eight columns a thread, eight threads a scale: a wave takes eight groups of
// one token at a time, kUnder such pieces of its tokens under way together.
template <int kType, int kUnder>
__global__ __launch_bounds__(kRowThreads) void kv_append_kernel(KvView kv, coli_moe_kv_rows_t r,
                                                                coli_moe_kv_values_t a, int parts) {
  const int lane = threadIdx.x & 63, D = kv.p.head_dim, ng = D / kKvGroup;
  const int groups = 2 * kv.p.kv_heads * ng, steps = (groups + 7) / 8;
  const int64_t waves = (int64_t)gridDim.x * (kRowThreads / 64);
  const int64_t work = (int64_t)((r.tokens + kGroup - 1) / kGroup) * parts;
  for (int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + uniform(threadIdx.x >> 6); w < work; w += waves) {
    const int t0 = (int)(w / parts) * kGroup, count = min(kGroup, r.tokens - t0);
    Located at;
    bool located = false;
    for (int n0 = (int)(w % parts) * kUnder; n0 < count * steps; n0 += parts * kUnder) {
      Raw8 raw[kUnder];
      // which group a lane has of piece n0 + u: its token, and 0 .. groups - 1 of keys and values
      auto group_of = [&](int u) { return (n0 + u) % steps * 8 + lane / 8; };
      auto token_of = [&](int u) { return min((n0 + u) / steps, count - 1); };
#pragma unroll
      for (int u = 0; u < kUnder; ++u) {
        const int gi = min(group_of(u), groups - 1), is_v = gi >= groups / 2, hg = gi - (is_v ? groups / 2 : 0);
        const int64_t t = t0 + token_of(u);
        const int h = hg / ng, col = hg % ng * kKvGroup + (lane & 7) * 8;
        raw[u] = load_raw8(is_v ? a.v : a.k, kType,
                           is_v ? t * a.v_token + h * a.v_head + col : t * a.k_token + h * a.k_head + col);
      }
      // looked up while the first values are on their way
      if (!located) at = locate(kv, r, t0);
      located = true;
#pragma unroll
      for (int u = 0; u < kUnder; ++u) {
        const int token = token_of(u);
        const int page = __builtin_amdgcn_readlane(at.page, token), slot = __builtin_amdgcn_readlane(at.slot, token);
        float x[8];
        unpack8(kType, raw[u], x);
        // as integers: Inf and NaN are above every finite value
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        top = max(top, (uint32_t)dpp_i<kDppQuadXor1>((int)top));
        top = max(top, (uint32_t)dpp_i<kDppQuadXor2>((int)top));
        top = max(top, (uint32_t)__shfl_xor((int)top, 4));
        const int gi = group_of(u);
        if (gi >= groups || n0 + u >= count * steps || page < 0) continue;
        const bool is_v = gi >= groups / 2;
        const int hg = is_v ? gi - groups / 2 : gi, h = hg / ng, g = hg % ng, col = g * kKvGroup + (lane & 7) * 8;
        // the quotient in float32 never falls on a bfloat16 border that the exact one is not on
        const uint16_t sb = top >= 0x7F800000u ? 0x7FC0 : to_bf16(__uint_as_float(top) / 7.0f);
        float sc = from_bf16(sb);
        uint32_t codes = 0;
        if (sc > 0.0f) {
          // away from the scales whose reciprocal overflows
          const float up = sc < 0x1p-100f ? 0x1p64f : 1.0f;
          sc *= up;
          const float rc = __builtin_amdgcn_rcpf(sc);
#pragma unroll
          for (int j = 0; j < 8; ++j) codes |= (uint32_t)(code4(x[j] * up, sc, rc) & 15) << (4 * j);
        }
        const uint64_t row = code_row(kv, page, h, slot);
        *reinterpret_cast<uint32_t *>((is_v ? kv.p.v_codes : kv.p.k_codes) + row * (D / 2) + col / 2) = codes;
        if ((lane & 7) == 0) {
          (is_v ? kv.p.v_scales : kv.p.k_scales)[(((int64_t)page * kv.p.kv_heads + h) * ng + g) * kv.p.page_size +
                                                 slot] = sb;
          if (kv.p.weights && g == 0 && !is_v) kv.p.weights[row] = 0.0f;
        }
      }
    }
  }
}

// Eight columns a thread; a wave takes 512 columns of one token at a time,
// kUnder such pieces of its tokens under way together.
template <int kType, int kUnder>
__global__ __launch_bounds__(kRowThreads) void kv_read_kernel(KvView kv, coli_moe_kv_rows_t r, coli_moe_kv_values_t a,
                                                              int parts) {
  const int lane = threadIdx.x & 63, D = kv.p.head_dim, ng = D / kKvGroup;
  const int units = 2 * kv.p.kv_heads * (D / 8), steps = (units + 63) / 64;
  const int64_t waves = (int64_t)gridDim.x * (kRowThreads / 64);
  const int64_t work = (int64_t)((r.tokens + kGroup - 1) / kGroup) * parts;
  for (int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + uniform(threadIdx.x >> 6); w < work; w += waves) {
    const int t0 = (int)(w / parts) * kGroup, count = min(kGroup, r.tokens - t0);
    const Located at = locate(kv, r, t0);
    for (int n0 = (int)(w % parts) * kUnder; n0 < count * steps; n0 += parts * kUnder) {
      int code[kUnder];
      uint16_t scale[kUnder];
      auto unit_of = [&](int u) { return (n0 + u) % steps * 64 + lane; };
      auto token_of = [&](int u) { return min((n0 + u) / steps, count - 1); };
#pragma unroll
      for (int u = 0; u < kUnder; ++u) {
        const int token = token_of(u), page = max(__builtin_amdgcn_readlane(at.page, token), 0);
        const int slot = __builtin_amdgcn_readlane(at.slot, token);
        const int n = min(unit_of(u), units - 1), is_v = n >= units / 2, hu = n - (is_v ? units / 2 : 0);
        const int h = hu / (D / 8), col = hu % (D / 8) * 8;
        code[u] = *reinterpret_cast<const int *>((is_v ? kv.p.v_codes : kv.p.k_codes) +
                                                 code_row(kv, page, h, slot) * (D / 2) + col / 2);
        scale[u] = (is_v ? kv.p.v_scales : kv.p.k_scales)[(((int64_t)page * kv.p.kv_heads + h) * ng + col / kKvGroup) *
                                                              kv.p.page_size + slot];
      }
#pragma unroll
      for (int u = 0; u < kUnder; ++u) {
        const int token = token_of(u), page = __builtin_amdgcn_readlane(at.page, token);
        const bool in_seq = __builtin_amdgcn_readlane((int)at.in_seq, token);
        const int n = unit_of(u);
        if (n >= units || n0 + u >= count * steps || !(in_seq || a.clear)) continue;
        const bool is_v = n >= units / 2;
        const int hu = is_v ? n - units / 2 : n, h = hu / (D / 8), col = hu % (D / 8) * 8;
        const float sc = page >= 0 ? from_bf16(scale[u]) : 0.0f;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = page >= 0 ? (float)((code[u] << (28 - 4 * j)) >> 28) * sc : 0.0f;
        const int64_t t = t0 + token;
        void *out = is_v ? a.v : a.k;
        const int64_t to = is_v ? t * a.v_token + h * a.v_head + col : t * a.k_token + h * a.k_head + col;
        if constexpr (kUnder > 1)
          store8_past(out, kType, to, 8, x);
        else
          store8(out, kType, to, x);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Eviction
// ---------------------------------------------------------------------------

constexpr int kSelectThreads = 1024;
constexpr int kSelectRows = 32768;  // rows whose keys LDS holds; those beyond are looked up each time

// Weights in an order of unsigned integers: larger weights larger, NaN above
// everything, -0 as 0.
__device__ __forceinline__ uint32_t rank_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A row that does not exist is below every weight.
__device__ __forceinline__ uint32_t row_key(const KvView &kv, const int32_t *table, int width, int h, int row) {
  const int page = row_page(kv, table, width, row);
  if (page < 0) return 0;
  return rank_key(kv.p.weights[code_row(kv, page, h, row & (kv.p.page_size - 1))]);
}

// The row that `rank` rows that exist stand before, of the sequence's first len;
// called by whole waves.
__device__ int row_of_rank(const KvView &kv, const int32_t *table, int width, int len, int rank) {
  const int lane = threadIdx.x & 63, pages = (len + kv.p.page_size - 1) >> kv.shift;
  int left = rank >> kv.shift;  // pages that exist, before the row's
  for (int i0 = 0; i0 < pages; i0 += 64) {
    const int i = i0 + lane;
    const bool there = i < pages && row_page(kv, table, width, (int64_t)i << kv.shift) >= 0;
    const uint64_t mask = __ballot(there);
    const int n = __popcll(mask);
    if (left < n) {
      const uint64_t it = __ballot(there && __popcll(mask & ((1ull << lane) - 1)) == left);
      return min(((i0 + __builtin_ctzll(it)) << kv.shift) + (rank & (kv.p.page_size - 1)), len);
    }
    left -= n;
  }
  return len;
}

// The rows that one sequence's key head keeps: the c-th largest key of the
// middle rows is found digit by digit (8 bits, largest first), then rows are
// kept while they are first, recent, above it, or among the first of those
// equal to it; each thread has rows side by side, so one sum over the
// workgroup places them.  Rows that do not exist are none of these: the first
// and the recent are counted among those that do.  Bound by the latency of its
// steps: every wave adds up a digit's counts for itself, so that a digit is one
// barrier.  600 rows 8 us, 16 sequences of up to 8192 rows, 8 heads, 19 us.
// (Counting a wave's equal digits together before LDS is asked: 35.)
__global__ __launch_bounds__(kSelectThreads) void kv_select_kernel(KvView kv, coli_moe_kv_rows_t r,
                                                                   coli_moe_kv_evict_t a) {
  constexpr int kWaves = kSelectThreads / 64;
  __shared__ uint32_t keys[kSelectRows];
  __shared__ int hist[4][256];
  __shared__ int2 sums[kWaves];
  __shared__ int lost[2][kWaves];
  static_assert(4 * 256 == kSelectThreads, "a count a thread");
  const int H = kv.p.kv_heads, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int turn = 0;
  for (int64_t w = blockIdx.x; w < (int64_t)r.seqs * H; w += gridDim.x) {
    const int s = (int)(w / H), h = (int)(w % H);
    const int32_t *table = r.table + s * r.table_stride;
    // lengths may be anything; at most 2^30 rows stand in a table
    const int len = min(max(r.lengths[s], 0), r.table_width << kv.shift);
    // rows among them that do not exist
    int gone = 0;
    for (int i = tid << kv.shift; i < len; i += kSelectThreads << kv.shift)
      if (row_page(kv, table, r.table_width, i) < 0) gone += min(kv.p.page_size, len - i);
    if (__any(gone > 0))
#pragma unroll
      for (int d = 1; d < 64; d *= 2) gone += __shfl_xor(gone, d);
    if (lane == 0) lost[turn][wave] = gone;
    __syncthreads();  // and of the item before, all is read
    gone = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) gone += lost[turn][i];
    turn ^= 1;
    const int have = len - gone;
    const int keep = min(a.keep, have);
    int32_t *kept = a.kept + w * a.keep;
    if (h == 0 && tid == 0) a.new_lengths[s] = keep;
    for (int i = keep + tid; i < a.keep; i += kSelectThreads) kept[i] = -1;
    if (len <= a.keep && gone == 0) {
      for (int i = tid; i < keep; i += kSelectThreads) kept[i] = i;
      continue;
    }
    // the middle: rows lo .. hi - 1
    int lo = a.first, hi = len - a.recent;
    if (__builtin_expect(gone > 0, 0)) {
      lo = have > a.keep ? row_of_rank(kv, table, r.table_width, len, a.first) : len;
      hi = have > a.keep ? row_of_rank(kv, table, r.table_width, len, have - a.recent) : len;
    }
    int need = have > a.keep ? keep - a.first - a.recent : 0;  // of the middle rows that exist, fewer than there are
    const bool any = need > 0;
    uint32_t key = 0, known = 0;  // digits found so far, and their mask
    auto key_of = [&](int row) {
      return row - lo < kSelectRows ? keys[row - lo] : row_key(kv, table, r.table_width, h, row);
    };
    if (any) {
      (&hist[0][0])[tid] = 0;
      // four lookups under way together
      const int held = min(hi - lo, kSelectRows);
      for (int i0 = tid; i0 < held; i0 += 4 * kSelectThreads) {
        uint32_t k[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          k[u] = row_key(kv, table, r.table_width, h, lo + min(i0 + u * kSelectThreads, held - 1));
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (i0 + u * kSelectThreads < held) keys[i0 + u * kSelectThreads] = k[u];
      }
      __syncthreads();
      for (int n = 0; n < 4; ++n) {
        const int shift = 24 - 8 * n;
        for (int row = lo + tid; row < hi; row += kSelectThreads) {
          const uint32_t k = key_of(row);
          if ((k & known) == key) atomicAdd(&hist[n][(k >> shift) & 255], 1);
        }
        __syncthreads();
        // digits from the largest down, four a lane, and the rows in them and above
        int count[4], upto = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) upto += count[i] = hist[n][255 - 4 * lane - i];
        const int own = upto;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
          const int y = __shfl_up(upto, d);
          if (lane >= d) upto += y;
        }
        const int at = __builtin_ctzll(__ballot(upto >= need) | 1ull << 63);
        int digit = 255 - 4 * lane, rest = need - (upto - own);
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (digit == 255 - 4 * lane - i && rest > count[i]) {
            rest -= count[i];
            --digit;
          }
        key |= (uint32_t)__builtin_amdgcn_readlane(digit, at) << shift;
        known |= 255u << shift;
        need = __builtin_amdgcn_readlane(rest, at);
      }
    }
    // need: rows equal to `key` still to take, in order
    const int each = (len + kSelectThreads - 1) / kSelectThreads;
    const int from = min(tid * each, len), to = min(from + each, len);
    auto outside = [&](int row) {  // the first and the recent ones
      return (row < lo || row >= hi) && (gone == 0 || row_page(kv, table, r.table_width, row) >= 0);
    };
    int same = 0, above = 0;
    for (int row = from; row < to; ++row) {
      const bool middle = row >= lo && row < hi;
      const uint32_t k = middle && any ? key_of(row) : 0;
      same += middle && any && k == key ? 1 : 0;
      above += outside(row) || (any && k > key) ? 1 : 0;
    }
    // of the threads before this one
    int rank = same, at = above;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int x = __shfl_up(rank, d), y = __shfl_up(at, d);
      if (lane >= d) rank += x, at += y;
    }
    if (lane == 63) sums[wave] = make_int2(rank, at);
    __syncthreads();
    rank -= same, at -= above;
    for (int i = 0; i < wave; ++i) rank += sums[i].x, at += sums[i].y;
    at += min(rank, need);  // those equal that were taken
    for (int row = from; row < to; ++row) {
      const bool middle = row >= lo && row < hi;
      const uint32_t k = middle && any ? key_of(row) : 0;
      const bool equal = middle && any && k == key;
      if (outside(row) || (any && k > key) || (equal && rank < need)) kept[at++] = row;
      rank += equal ? 1 : 0;
    }
  }
}

// Copies the kept rows: 16 bytes a thread, rows of one head side by side.
// Bound by bytes: 61575 rows of 8 heads of 128, 138 MB: 26 us (5.3 TB/s).
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

// Waves of a token group's pieces: one piece each where that does not fill the
// chip twice, else as many waves of four pieces as do, or one.  (4889 tokens, 4
// heads of 256, append and read: one round of waves 30 us, four rounds 35; pieces
// by two or eight 34.  One piece a wave for 64 tokens: append 5 us, by four 12.)
struct Parts {
  int under, parts;
};
Parts parts_of(int tokens, int steps) {
  const int64_t groups = (tokens + kGroup - 1) / kGroup, fill = 16384 / groups;
  const int pieces = (tokens < kGroup ? tokens : kGroup) * steps, fours = (pieces + 3) / 4;
  if (pieces <= fill) return {1, pieces};
  return {4, (int)(fill < 1 ? 1 : fours < fill ? fours : fill)};
}

using RowsKernel = void (*)(KvView, coli_moe_kv_rows_t, coli_moe_kv_values_t, int);

template <int kUnder>
RowsKernel append_of(int type) {
  return type == COLI_MOE_F32    ? kv_append_kernel<COLI_MOE_F32, kUnder>
         : type == COLI_MOE_BF16 ? kv_append_kernel<COLI_MOE_BF16, kUnder>
                                 : kv_append_kernel<COLI_MOE_F16, kUnder>;
}
template <int kUnder>
RowsKernel read_of(int type) {
  return type == COLI_MOE_F32    ? kv_read_kernel<COLI_MOE_F32, kUnder>
         : type == COLI_MOE_BF16 ? kv_read_kernel<COLI_MOE_BF16, kUnder>
                                 : kv_read_kernel<COLI_MOE_F16, kUnder>;
}

hipError_t launch_rows(RowsKernel kernel, const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r,
                       const coli_moe_kv_values_t &a, const Parts &p, hipStream_t s) {
  const int64_t waves = (int64_t)((r.tokens + kGroup - 1) / kGroup) * p.parts;
  return launch(kernel, dim3(grid_of((waves + kRowThreads / 64 - 1) / (kRowThreads / 64))), dim3(kRowThreads), 0, s,
                kv_view(kv), r, a, p.parts);
}

}  // namespace

hipError_t launch_kv_append(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_values_t &a,
                            hipStream_t s) {
  const Parts p = parts_of(r.tokens, (2 * kv.kv_heads * (kv.head_dim / kKvGroup) + 7) / 8);
  return launch_rows(p.under == 1 ? append_of<1>(a.type) : append_of<4>(a.type), kv, r, a, p, s);
}

hipError_t launch_kv_read(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_values_t &a,
                          hipStream_t s) {
  const Parts p = parts_of(r.tokens, (2 * kv.kv_heads * (kv.head_dim / 8) + 63) / 64);
  return launch_rows(p.under == 1 ? read_of<1>(a.type) : read_of<4>(a.type), kv, r, a, p, s);
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
