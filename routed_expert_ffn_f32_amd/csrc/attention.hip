// Attention over the paged 4-bit cache (coli_moe_kv_attention).
//
// One tile of work is 16 columns of a 16x16x32 half-precision matrix
// instruction: a column is a query row (a query head of one token) together
// with one 64-column group of the head, so that each column has its own scale
// of the keys and of the values and the codes themselves can be the operands.
// With D = 128 that is 8 rows times 2 groups.
//
//  - scores, transposed: A = codes of 16 keys, B = the query, zero outside the
//    column's group; the column's key scale is applied to the sum, and the
//    groups of a row are added across lanes (a rotation within 16 lanes).
//  - values, transposed: A = codes of 16 columns' values for 32 keys, B = the
//    softmax weights times the column's value scale.  The weights come out of
//    the scores in the layout that B wants.
//
// Codes become halves exactly, in place: u = code ^ 8 is 8 more than the signed
// code; its four bits at the bottom of the half 1024 read 1024 + u (at bit 4:
// 1024 + 16 u), and one packed addition (fma) leaves u - 8.  (The bits alone,
// as subnormal halves, need no addition, but the matrix core aligns its
// products by exponents that it does not normalise: next to a large product
// everything below 2^-17 of it was lost.)
//
// A weight times its scale is rounded to the 11 bits of a half (results of 8
// bits, bfloat16) or to two halves' 22 (results of 11, half precision).
//
// Bound by bytes where there are many keys, 136 of a key head of 128 columns
// for one query: a decode batch of 64 sequences of up to 8192 rows, 8 key heads
// for 64 queries, 327 MB, takes 91 us (3.6 TB/s; a large copy 5.1) with a
// workgroup for each sequence's key head and no join, one sequence of 131071
// rows, 143 MB, 42 us, 5 of them the join.  What keeps it from the copy's rate is
// the 350 vector instructions of a step of 32 keys (columns are only 8 rows, so
// the expansion of codes has few to be shared by).  One sequence of 517 rows
// takes 14 us: a launch, three loads that follow each other (length, page, rows),
// three steps a wave and the join of eight waves.
#include "attention.h"
#include "lds_dma.h"

namespace coli {
namespace {

template <int D>
struct Tile {
  static constexpr int kGroups = D / kKvGroup;
  static constexpr int kRows = 16 / kGroups;       // query rows of a tile
  static constexpr int kSteps = D / 32;            // matrix instructions of 16 keys' scores
  static constexpr int kParts = D / 16;            // of 32 keys' values
  static constexpr int kWords = D == 256 ? 2 : 1;  // dwords of a key's values that a lane holds
  // A step in LDS: codes of 32 keys and of their values as in memory, then the
  // scales, 64 bytes for each group of the keys and then of the values.
  static constexpr int kCodes = 16 * D;            // bytes of the keys, and of the values
  static constexpr int kScales = 2 * kCodes;       // where the scales start
  static constexpr int kCopies = 2 * D / 64 + (D == 256 ? 2 : 1);  // instructions that fetch a step
  static constexpr int kStep = kScales + (D == 256 ? 512 : 256);
  static constexpr int kRing = D == 64 ? 4 : D == 128 ? 3 : 2;     // steps a wave has room for
};
constexpr int kStepKeys = 32;  // keys of one step of a wave

// The larger of (sum over) a column's four lanes.
__device__ __forceinline__ float max_over_j(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_j(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
// Over the groups of a row: every lane of the row's columns gets it.
template <int D>
__device__ __forceinline__ float sum_groups(float v) {
  if constexpr (D >= 128) v += dpp_row_f<kDppRowRor8>(v);
  if constexpr (D >= 256) v += dpp_row_f<kDppRowRor4>(v);
  return v;
}
template <int D>
__device__ __forceinline__ float max_groups(float v) {
  if constexpr (D >= 128) v = fmaxf(v, dpp_row_f<kDppRowRor8>(v));
  if constexpr (D >= 256) v = fmaxf(v, dpp_row_f<kDppRowRor4>(v));
  return v;
}

// The column of this lane: its group, and the query row it stands for.
struct Column {
  int g, row;   // group; row of the sequence's key head (query * group + head)
  bool live;
  int token, head;
  int lo, hi;   // first and last row of the cache that the query sees
};

template <int D>
__device__ __forceinline__ Column column_of(const Call &c, SeqSpan span, int64_t len, int h, int tile) {
  const int col = threadIdx.x & 15;
  Column q;
  q.g = col / Tile<D>::kRows;
  q.row = tile * Tile<D>::kRows + col % Tile<D>::kRows;
  q.live = q.row < span.n * c.group;
  const int i = q.live ? q.row / c.group : 0;
  q.token = span.first + i;
  q.head = h * c.group + (q.live ? q.row % c.group : 0);
  const int64_t pos = len - span.n + i;
  q.hi = (int)min(max(pos, (int64_t)-1), (int64_t)1 << 30);
  q.lo = c.a.window ? (int)min(max(pos - c.a.window + 1, (int64_t)0), (int64_t)1 << 30) : 0;
  return q;
}

// The query operand of a column: exact in half precision after a power of two
// per row (elements below 2^-28 of the row's largest are rounded).  The sign of
// the call's scale goes with it and a scale of 0 makes it 0, so that what
// multiplies a score is positive.
template <int D>
struct QueryOperand {
  half8_t b[Tile<D>::kSteps];
  float unit;  // that takes the power of two back
};

template <int D>
__device__ __forceinline__ void load_query(const Call &c, const Column &q, QueryOperand<D> &f) {
  constexpr int kSteps = Tile<D>::kSteps;
  const int j = (threadIdx.x >> 4) & 3;
  u32x4 raw[kSteps];
  float top = 0.0f;
  const uint16_t *row = static_cast<const uint16_t *>(c.a.q) + (q.token * c.a.q_token + q.head * c.a.q_head);
#pragma unroll
  for (int w = 0; w < kSteps; ++w) {
    // columns of dword w of this lane: D = 64 has two a lane, D = 256 two sets of four
    const int col = D == 64 ? 16 * j + 8 * w : D == 128 ? 32 * j + 8 * w : 128 * (w / 4) + 32 * j + 8 * (w % 4);
    raw[w] = u32x4{0, 0, 0, 0};
    if (q.live && col / kKvGroup == q.g) raw[w] = load16(reinterpret_cast<const char *>(row + col));
  }
  const int type = c.a.type;
#pragma unroll
  for (int w = 0; w < kSteps; ++w) {
    float v[8];
    unpack8(type, Raw8{raw[w], raw[w]}, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
  }
  top = max_groups<D>(max_over_j(top));
  const int ex = lift_exponent(top);
  const float up = c.a.scale > 0.0f ? lift(ex) : c.a.scale < 0.0f ? -lift(ex) : 0.0f;
#pragma unroll
  for (int w = 0; w < kSteps; ++w) {
    float v[8];
    unpack8(type, Raw8{raw[w], raw[w]}, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f.b[w][2 * e] = (_Float16)(v[e] * up);
      f.b[w][2 * e + 1] = (_Float16)(v[e + 4] * up);
    }
  }
  f.unit = unlift(ex);
}

// Four neighbouring scales of a column's group.
__device__ __forceinline__ float4_t scales4(uint2 v) {
  return float4_t{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                  __uint_as_float(v.y & 0xFFFF0000u)};
}

// Keys and values of a step as they stand in memory.  Keys: lane (r, j) has
// columns of key r of each 16 (see load_query) and the scales of its column's
// group for keys 4 j ..  Values: lane (r, j) has, of keys 4 j .. 4 j + 3 of each
// 16, the dword of columns 8 r .. 8 r + 7, and the same scales.
template <int D>
struct KeyRegs {
  u32x4 k[2][D == 256 ? 2 : 1];
  uint2 s[2];
};
template <int D>
struct ValueRegs {
  uint32_t v[2][4][Tile<D>::kWords];
  uint2 s[2];
};

template <int D, bool kSmallPages>
__device__ __forceinline__ void load_keys(const Call &c, const Place<kSmallPages> &p, int g, KeyRegs<D> &r) {
  const int lane = threadIdx.x & 63, j = lane >> 4;
  const uint32_t row = (lane & 15) * (D / 2) + (D == 64 ? 8 : 16) * j, scale = (g << c.kv.shift) + 4 * j;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int n = kSmallPages ? t : 0, rows = kSmallPages ? 0 : 16 * t;
    const uint8_t *base = c.kv.p.k_codes + p.row[n] * (D / 2);
    if constexpr (D == 64) {
      const uint2 v = *reinterpret_cast<const uint2 *>(base + row + rows * (D / 2));
      r.k[t][0] = u32x4{v.x, v.y, 0, 0};
    } else {
#pragma unroll
      for (int w = 0; w < D / 128; ++w)
        r.k[t][w] = *reinterpret_cast<const u32x4 *>(base + row + (rows * (D / 2) + 64 * w));
    }
    r.s[t] = *reinterpret_cast<const uint2 *>(c.kv.p.k_scales + p.scale[n] + scale + rows);
  }
}

// An infinite scale counts as NaN: its products are Inf or 0, which a maximum
// or a weight of 0 would hide.
__device__ __forceinline__ float finite_or_nan(float v) { return fabsf(v) == INFINITY ? NAN : v; }

// A query's lifted products with codes are up to 2^27, so scales from 2^100 on
// may take them past float32's range although the scores are within it.  Such a
// step's scales are multiplied by this first and its scores by the inverse
// afterwards; queries so large that the inverse would pass the range itself
// have scores within it only with scales that need no care.
constexpr float kDown = 0x1p-27f;
__device__ __forceinline__ float scores_down(float unit) { return unit < 0x1p100f ? kDown : 1.0f; }
__device__ __forceinline__ float odd_unit(float unit) { return unit < 0x1p100f ? unit * (1 / kDown) : unit; }

// Scores of 16 keys, to be multiplied by the operand's unit: lane (column, j)
// gets keys 4 j .. 4 j + 3.  kOdd: some scales of the keys may be infinite or
// above 2^100, and what the scores are to be multiplied by is odd_unit.
template <int D, bool kOdd = false>
__device__ __forceinline__ float4_t scores16(const KeyRegs<D> &r, int t, const QueryOperand<D> &f) {
  float4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < Tile<D>::kSteps; ++w)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_of(r.k[t][w / 4][w % 4]), f.b[w], acc, 0, 0, 0);
  const float4_t sc = scales4(r.s[t]);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc[i] = sum_groups<D>(acc[i] * (kOdd ? finite_or_nan(sc[i]) * scores_down(f.unit) : sc[i]));
  return acc;
}

// Zeros in the out rows of tokens that no sequence has.
__device__ __forceinline__ void clear_outside(const Call &c, int D) {
  if (!c.a.clear || !c.rows.offsets) return;
  const int T = c.rows.tokens;
  const int first = min(max(c.rows.offsets[0], 0), T), last = min(max(c.rows.offsets[c.rows.seqs], first), T);
  const int64_t gap = first + (int64_t)(T - last), per = (int64_t)c.a.q_heads * D;
  for (int64_t i = threadIdx.x; i < gap * per; i += blockDim.x) {
    const int64_t n = i / per, e = i % per;
    const int64_t t = n < first ? n : last + (n - first);
    static_cast<uint16_t *>(c.a.out)[t * c.a.out_token + e / D * c.a.out_head + e % D] = 0;
  }
}

// weights_out = weights for the rows that a query sees, where the sums are not
// added to the cache's own weights: part `item` of the sequences' key heads.  A
// place may belong to several sequences, so this is done before any sum is
// added, by workgroups of the attention's own launch (a launch of its own: 4 us
// more).
__device__ __forceinline__ void copy_weights(const Call &c, int64_t item) {
  const int H = c.kv.p.kv_heads, parts = c.copy_parts;
  const int h = (int)(item / parts % H), s = (int)(item / parts / H);
  const SeqSpan span = seq_span(c.rows, s);
  if (span.n == 0) return;
  const int64_t len = c.rows.lengths[s], lo = c.a.window ? max(len - span.n - c.a.window + 1, (int64_t)0) : 0;
  const int64_t end = min(len, (int64_t)c.rows.table_width << c.kv.shift);
  const int32_t *table = c.rows.table + s * c.rows.table_stride;
  const int64_t step = (int64_t)parts * (4 * blockDim.x);  // four rows a thread, within a page
  for (int64_t key = (item % parts * blockDim.x + threadIdx.x) * 4; key < end; key += step) {
    const int page = row_page(c.kv, table, c.rows.table_width, key);
    if (page < 0 || key + 4 <= lo) continue;
    const uint64_t at = code_row(c.kv, page, h, (int)key & (c.kv.p.page_size - 1));
    const float4_t w = *reinterpret_cast<const float4_t *>(c.kv.p.weights + at);
    if (key >= lo && key + 4 <= len) {
      *reinterpret_cast<float4_t *>(c.a.weights_out + at) = w;
      continue;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (key + i >= lo && key + i < len) c.a.weights_out[at + i] = w[i];
  }
}

// Weights times scales are lifted to [2^6, 2^7) at a weight of 1 and may pass
// it by the 2^kSlack that scores may pass the maximum by: 2^15 at most.
__device__ __forceinline__ float weight_lift(int ex) { return __uint_as_float((uint32_t)(260 - ex) << 23); }
__device__ __forceinline__ float weight_unlift(int ex) { return __uint_as_float((uint32_t)(ex - 6) << 23); }

// Copies a step's codes and scales into LDS.
template <int D, bool kSmallPages>
__device__ __forceinline__ void fetch_step(const Call &c, const Place<kSmallPages> &p, uint32_t lds) {
  using T = Tile<D>;
  const uint32_t lane = threadIdx.x & 63;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint8_t *codes = kv ? c.kv.p.v_codes : c.kv.p.k_codes;
    const uint32_t to = lds + kv * T::kCodes;
    if constexpr (D == 64 && kSmallPages) {
      const uint8_t *lo = codes + p.row[0] * (D / 2), *hi = codes + p.row[kSmallPages ? 1 : 0] * (D / 2);
      dma16v(to, (lane < 32 ? lo : hi) + (lane & 31) * 16);
    } else {
#pragma unroll
      for (int n = 0; n < D / 64; ++n) {  // 1024 bytes each: within 16 keys, but for D = 64
        constexpr int kEach = D >= 128 ? D / 128 : 1;  // of 16 keys
        const int t = kSmallPages ? n / kEach : 0, at = kSmallPages ? n % kEach : n;
        dma16(to + n * 1024, codes + p.row[kSmallPages ? t : 0] * (D / 2) + at * 1024, lane * 16);
      }
    }
  }
  // 16 lanes a group, two scales each
#pragma unroll
  for (int n = 0; n < (D == 256 ? 2 : 1); ++n) {
    const uint32_t seg = lane / 16, g = D == 64 ? 0 : D == 128 ? seg & 1 : seg;
    const bool values = D == 64 ? seg & 1 : D == 128 ? seg >> 1 : n == 1;
    const uint16_t *scales = values ? c.kv.p.v_scales : c.kv.p.k_scales;
    const uint64_t first = kSmallPages && (lane & 8) ? p.scale[kSmallPages ? 1 : 0] : p.scale[0];
    dma4v(lds + T::kScales + n * 256,
          scales + first + (g << c.kv.shift) + (kSmallPages ? lane & 7 : lane & 15) * 2);
  }
}

template <int D>
__device__ __forceinline__ void read_keys(const char *step, int g, KeyRegs<D> &r) {
  const int lane = threadIdx.x & 63, j = lane >> 4;
  const char *row = step + (lane & 15) * (D / 2) + (D == 64 ? 8 : 16) * j;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    if constexpr (D == 64) {
      const uint2 v = *reinterpret_cast<const uint2 *>(row + 16 * t * (D / 2));
      r.k[t][0] = u32x4{v.x, v.y, 0, 0};
    } else {
#pragma unroll
      for (int w = 0; w < D / 128; ++w) r.k[t][w] = *reinterpret_cast<const u32x4 *>(row + 16 * t * (D / 2) + 64 * w);
    }
    r.s[t] = *reinterpret_cast<const uint2 *>(step + Tile<D>::kScales + 64 * g + 32 * t + 8 * j);
  }
}

// Of two scales: the sign's bits are those that are NaN, Inf or from 2^100 on.
__device__ __forceinline__ uint32_t odd_bits(uint32_t two) { return (two & 0x7FFF7FFFu) + 0x0E800E80u; }
// Whether one of a step's scales is, of the keys or of the values: a lane looks
// at two (D = 256: four).
template <int D>
__device__ __forceinline__ bool scales_odd(const char *step) {
  const char *at = step + Tile<D>::kScales + (threadIdx.x & 63) * (D == 256 ? 8 : 4);
  uint32_t v = odd_bits(*reinterpret_cast<const uint32_t *>(at));
  if constexpr (D == 256) v |= odd_bits(*reinterpret_cast<const uint32_t *>(at + 4));
  return __any((v & 0x80008000u) != 0);
}
// The same of a step's keys in registers.
template <int D>
__device__ __forceinline__ bool keys_odd(const KeyRegs<D> &r) {
  const uint32_t v = odd_bits(r.s[0].x) | odd_bits(r.s[0].y) | odd_bits(r.s[1].x) | odd_bits(r.s[1].y);
  return __any((v & 0x80008000u) != 0);
}

template <int D>
__device__ __forceinline__ void read_values(const char *step, int g, ValueRegs<D> &r) {
  using T = Tile<D>;
  const int lane = threadIdx.x & 63, j = lane >> 4;
  const char *word =
      step + T::kCodes + 4 * j * (D / 2) + (D == 64 ? (lane & 15) / 2 * 4 : (lane & 15) * 4);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int w = 0; w < T::kWords; ++w)
        r.v[t][i][w] = *reinterpret_cast<const uint32_t *>(word + (16 * t + i) * (D / 2) + 64 * w);
    r.s[t] = *reinterpret_cast<const uint2 *>(step + T::kScales + 64 * (T::kGroups + g) + 32 * t + 8 * j);
  }
}

// One workgroup: `tile_waves` tiles of one sequence's key head over one split
// of their keys; the waves of a tile take its steps of keys in turn and are
// joined in LDS at the end.  A wave copies its steps into a ring of its own in
// LDS, up to kRing - 1 ahead.  kTwice: the weights as the sum of two halves.
template <int D, bool kTwice, bool kSmallPages, int kWaves>
__global__ __launch_bounds__(64 * kWaves, D == 256 || kWaves == 8 ? 2 : D == 128 ? 3 : 4) void kv_attention_kernel(
    Call c, int64_t work) {
  using T = Tile<D>;
  constexpr int kOut = T::kRows * D;  // 1024
  constexpr int kThreads = 64 * kWaves;
  // the rings; at the end every wave's sums and results
  __shared__ __align__(16) char shared[kWaves * T::kRing * T::kStep];
  static_assert(T::kRing * T::kStep >= kOut * 4 + T::kRows * 8, "results fit where the ring was");
  float *so = reinterpret_cast<float *>(shared);                                // [wave][row][column]
  float2 *sml = reinterpret_cast<float2 *>(shared + kWaves * kOut * sizeof(float));  // [wave][row]
  const int tid = threadIdx.x, lane = tid & 63, j = lane >> 4, wave = uniform(tid >> 6);
  const int H = c.kv.p.kv_heads;
  if (blockIdx.x >= (unsigned)c.blocks) {
    const int64_t copies = (int64_t)c.rows.seqs * H * c.copy_parts;
    for (int64_t item = blockIdx.x - c.blocks; item < copies; item += gridDim.x - c.blocks) copy_weights(c, item);
    return;
  }
  const char *ring = shared + wave * T::kRing * T::kStep;
  const uint32_t ring_lds = uniform(lds_addr(ring));
  if (blockIdx.x == 0) clear_outside(c, D);
  for (int64_t item = blockIdx.x; item < work; item += c.blocks) {
    const int tgroups = c.tiles / c.tile_waves;
    const int tg = (int)(item % tgroups);
    const int64_t rest = item / tgroups;
    const int split = (int)(rest % c.splits), h = (int)(rest / c.splits % H), s = (int)(rest / c.splits / H);
    const SeqSpan span = seq_span(c.rows, s);
    const int rows = span.n * c.group, r0 = tg * c.tile_waves * T::kRows;
    if (r0 >= rows || rows > c.few_rows) continue;
    // a sequence of fewer rows than the call has room for: its keys are dealt to more waves
    const int tile_waves = rows <= T::kRows ? 1 : rows <= 2 * T::kRows ? min(c.tile_waves, 2) : c.tile_waves;
    const int64_t len = c.rows.lengths[s];
    const int32_t *table = c.rows.table + s * c.rows.table_stride;
    const int tile = tg * c.tile_waves + wave % tile_waves;
    const int kw = wave / tile_waves, kn = kWaves / tile_waves;
    const int r1 = min(r0 + tile_waves * T::kRows, rows) - 1;
    const KeyRange range = keys_of_rows(c, span, len, r0, r1);
    // keys are numbers up to 2^30
    const int begin = (int)min(range.lo, (int64_t)1 << 30) & ~(kStepKeys - 1), end = (int)max(range.hi, (int64_t)0);
    const int steps = range.hi > range.lo ? (end - begin + kStepKeys - 1) / kStepKeys : 0;
    const int per = max((steps + c.splits - 1) / c.splits, 2 * kn);  // a split has some work for each wave
    const int s0 = min(split * per, steps), s1 = min(s0 + per, steps);
    const int mine = s1 - s0 > kw ? (s1 - s0 - kw + kn - 1) / kn : 0;  // steps of this wave
    const int first_key = begin + (s0 + kw) * kStepKeys, key_step = kn * kStepKeys;

    const Column q = column_of<D>(c, span, len, h, tile);
    __syncthreads();  // of the item before, all is read
    // the table's entries of 64 steps at a time, a step a lane
    Entries<kSmallPages> entries;
    auto look_up = [&](int i) { entries = entries_of<kSmallPages>(c, table, first_key + min(i + lane, mine - 1) * key_step); };
    uint32_t there = 0;  // bit 2 slot + t: the 16 keys are on a page
    auto fetch = [&](int i, int slot) {
      const int key0 = first_key + i * key_step;
      Entries<kSmallPages> e;
#pragma unroll
      for (int t = 0; t < (kSmallPages ? 2 : 1); ++t) e.entry[t] = __builtin_amdgcn_readlane(entries.entry[t], i & 63);
      const Place<kSmallPages> p = place_of<D>(c, e, h, key0);
      there = (there & ~(3u << 2 * slot)) | (uint32_t)(p.ok[0] | p.ok[1] << 1) << 2 * slot;
      fetch_step<D>(c, p, ring_lds + slot * T::kStep);
    };
    if (mine > 0) {
      look_up(0);
#pragma unroll
      for (int i = 0; i < T::kRing - 1; ++i)
        if (i < mine) fetch(i, i);
    }
    QueryOperand<D> f;
    load_query<D>(c, q, f);
    // rows of this wave's tile alone, for steps that all of them see whole
    auto clamped = [](int64_t v) { return (int)min(max(v, (int64_t)-1), (int64_t)1 << 30); };
    const int64_t first_pos = len - span.n + min(tile * T::kRows, rows - 1) / c.group;
    const int64_t last_pos = len - span.n + min((tile + 1) * T::kRows - 1, rows - 1) / c.group;
    const int all_hi = clamped(first_pos), all_lo = c.a.window ? clamped(last_pos - c.a.window + 1) : 0;

    float m = -INFINITY, l = 0.0f;  // the maximum that the sums stand against; the sum
    bool far = false;               // a column's maximum is above kFar
    int ex = lift_exponent(0.0f);   // weights times scales are lifted by it
    float big = 0.0f;               // the largest of them, lifted
    float4_t acc[T::kParts];
#pragma unroll
    for (int i = 0; i < T::kParts; ++i) acc[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

    int slot = 0;
    for (int i = 0; i < mine; ++i) {
      // this step has come when only the later ones' copies are under way
      if (i + T::kRing - 1 <= mine)
        dma_wait<(T::kRing - 2) * T::kCopies>();
      else
        dma_wait<0>();
      const char *step = ring + slot * T::kStep;
      KeyRegs<D> kr;
      read_keys<D>(step, q.g, kr);
      const int key0 = first_key + i * key_step;
      const bool ok[2] = {(there >> 2 * slot & 1) != 0, (there >> 2 * slot & 2) != 0};
      if (i + T::kRing - 1 < mine) {
        // where the step before this one was
        const int ahead = i + T::kRing - 1, at = slot == 0 ? T::kRing - 1 : slot - 1;
        if ((ahead & 63) == 0) look_up(ahead);
        fetch(ahead, at);
      }
      float4_t x[2], sv[2];
      const bool odd = scales_odd<D>(step);
      float unit = f.unit;
#pragma unroll
      for (int t = 0; t < 2; ++t) x[t] = scores16<D>(kr, t, f);
      ValueRegs<D> vr;
      read_values<D>(step, q.g, vr);
#pragma unroll
      for (int t = 0; t < 2; ++t) sv[t] = scales4(vr.s[t]);
      if (__builtin_expect(!(key0 + kStepKeys - 1 <= all_hi && key0 >= all_lo && ok[0] && ok[1]) || odd, 0)) {
        if (odd) {
          KeyRegs<D> again;
          read_keys<D>(step, q.g, again);
#pragma unroll
          for (int t = 0; t < 2; ++t) x[t] = scores16<D, true>(again, t, f);
          unit = odd_unit(f.unit);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 16 * t + 4 * j + i;
            const bool seen = ok[t] && key <= q.hi && key >= q.lo;
            x[t][i] = seen ? x[t][i] : -INFINITY;
            sv[t][i] = seen ? finite_or_nan(sv[t][i]) : 0.0f;
          }
      }
      float top = x[0][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e / 4][e % 4]);
      top *= unit;
      float w[8], sum;
      auto weigh = [&]() {
        const float base = m == -INFINITY ? 0.0f : m, up = weight_lift(ex);
        float z[8];
        if (__builtin_expect(far, 0)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = __builtin_fmaf(x[e / 4][e % 4], unit, -base) * c.cs;
        } else {
          const float by = fmaxf(unit * c.cs, 0x1p-126f), less = base * c.cs;  // -Inf times by is -Inf
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = __builtin_fmaf(x[e / 4][e % 4], by, -less);
        }
        sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = __builtin_amdgcn_exp2f(z[e]);
          sum += p;
          w[e] = p * sv[e / 4][e % 4] * up;
        }
      };
      weigh();
      float most = big;
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(w[e]));
      if (__builtin_expect(__any((top - m) * c.cs > kSlack || most > 0x1p15f), 0)) {
        // a new maximum, and the lift by the largest weight times scale against it
        const float m1 = fmaxf(m, max_over_j(top)), base = m1 == -INFINITY ? 0.0f : m1;
        const float fade = __builtin_amdgcn_exp2f((m - base) * c.cs);
        m = m1;
        far = __any(fabsf(m) * c.cs > kFar && m != -INFINITY);
        most = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          most = fmaxf(most, fabsf(__builtin_amdgcn_exp2f(__builtin_fmaf(x[e / 4][e % 4], unit, -base) * c.cs) *
                                   sv[e / 4][e % 4]));
        most = fmaxf(max_over_j(most), max_over_j(big) * weight_unlift(ex) * fade);
        const int ex1 = lift_exponent(most);
        l *= fade;
#pragma unroll
        for (int i = 0; i < T::kParts; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_amdgcn_ldexpf(acc[i][e] * fade, ex - ex1);
        ex = ex1;
        most *= weight_lift(ex);
        weigh();
      }
      big = most;
      l += sum;

      half8_t b, b2;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        b[e] = (_Float16)w[e];
        if constexpr (kTwice) b2[e] = (_Float16)(w[e] - (float)b[e]);
      }
      // D = 64: a lane's four columns are one half of its dword
      const uint32_t half = D == 64 ? 0x00020002u * (lane & 1) : 0u;
#pragma unroll
      for (int i = 0; i < T::kParts; i += 2) {
        const uint32_t sel = (0x0C040C00u + 0x00010001u * (i / 2 % 4)) + half;
        u32x4 lo, hi;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t two =
              __builtin_amdgcn_perm(vr.v[e / 2][2 * (e % 2) + 1][i / 8], vr.v[e / 2][2 * (e % 2)][i / 8], sel);
          lo[e] = low_codes(two);
          hi[e] = high_codes(two);
        }
        const half8_t a0 = __builtin_bit_cast(half8_t, lo), a1 = __builtin_bit_cast(half8_t, hi);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, b, acc[i], 0, 0, 0);
        acc[i + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, b, acc[i + 1], 0, 0, 0);
        if constexpr (kTwice) {
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, b2, acc[i], 0, 0, 0);
          acc[i + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, b2, acc[i + 1], 0, 0, 0);
        }
      }
      slot = slot + 1 == T::kRing ? 0 : slot + 1;
    }

    // this wave's sums, against its maximum: to LDS
    l = sum_over_j(l);
    const float down = weight_unlift(ex);
    const int col = lane & 15, r = col % T::kRows;
    __syncthreads();  // all rings are read
    if (j == 0 && q.g == 0) sml[wave * T::kRows + r] = make_float2(m, l);
#pragma unroll
    for (int i = 0; i < T::kParts; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = D == 64 ? 16 * j + 4 * e + i : 128 * (i / 8) + 32 * j + 8 * e + i % 8;
        if (d / kKvGroup == q.g) so[wave * kOut + r * D + d] = acc[i][e] * down;
      }
    __syncthreads();
    for (int e = tid; e < tile_waves * kOut; e += kThreads) {
      const int tw = e / kOut, rr = e % kOut / D, d = e % D;
      const int row = r0 + tw * T::kRows + rr;
      if (row >= rows) continue;
      float mm = -INFINITY;
      for (int k = 0; k < kn; ++k) mm = fmaxf(mm, sml[(k * tile_waves + tw) * T::kRows + rr].x);
      const float base = mm == -INFINITY ? 0.0f : mm;
      float o = 0.0f, ll = 0.0f;
      for (int k = 0; k < kn; ++k) {
        const int wv = k * tile_waves + tw;
        const float2 v = sml[wv * T::kRows + rr];
        const float fade = __builtin_amdgcn_exp2f((v.x - base) * c.cs);
        ll += v.y * fade;
        o += so[wv * kOut + rr * D + d] * fade;
      }
      const int token = span.first + row / c.group, head = h * c.group + row % c.group;
      const int64_t id = (int64_t)token * c.a.q_heads + head;
      if (c.splits > 1) {
        c.part_o[(id * c.part_splits + split) * D + d] = o;
        if (d == 0) c.part_ml[id * c.part_splits + split] = make_float2(mm, ll);
      } else {
        store1(c.a.out, c.a.type, token * c.a.out_token + head * c.a.out_head + d, ll != 0.0f ? o / ll : 0.0f);
        if (d == 0 && c.ml) c.ml[id] = make_float2(mm, ll);
      }
    }
  }
}

// Joins the splits of a row: kJoin waves a row (1 or 4, for few rows of many
// splits), D / 64 columns a lane.  Where only sequences of few rows have
// splits, the rows are counted by sequence, else by token.
template <int D, int kJoin>
__global__ __launch_bounds__(kTileThreads) void kv_attention_join_kernel(Call c, int few, int64_t work) {
  constexpr int kCols = D / 64, kRowsEach = kTileWaves / kJoin;
  __shared__ float sums[kJoin > 1 ? kTileWaves : 1][D];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int part = wave % kJoin;
  const int64_t step = (int64_t)gridDim.x * kRowsEach;
  for (int64_t item = (int64_t)blockIdx.x * kRowsEach + wave / kJoin; item < work; item += step) {
    int token, head, splits = c.splits;
    if (few > 0) {
      const int i = (int)(item % few), h = (int)(item / few % c.kv.p.kv_heads), s = (int)(item / few / c.kv.p.kv_heads);
      const SeqSpan span = seq_span(c.rows, s);
      const int rows = span.n * c.group;
      if (i >= rows || rows > c.few_rows) continue;
      token = span.first + i / c.group;
      head = h * c.group + i % c.group;
    } else {
      token = (int)(item / c.a.q_heads);
      head = (int)(item % c.a.q_heads);
      const int s = find_seq(c.rows, token);
      if (s < 0) continue;
      if (seq_span(c.rows, s).n * c.group > c.few_rows) splits = c.prompt_splits;
      if (splits == 1) continue;
    }
    const int64_t id = (int64_t)token * c.a.q_heads + head;
    const float2 *ml = c.part_ml + id * c.part_splits;
    // a split a lane: at most 128
    float2 mine[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) mine[k] = lane + 64 * k < splits ? ml[lane + 64 * k] : make_float2(-INFINITY, 0.0f);
    // this wave's splits, eight under way at a time; the last one again past the end, times 0
    const int per = (splits + kJoin - 1) / kJoin, first = part * per, last = min(first + per, splits);
    const float *from = c.part_o + id * c.part_splits * D + lane * kCols;
    float v[8][kCols];
    auto load = [&](int k0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) __builtin_memcpy(v[k], from + (int64_t)min(k0 + k, splits - 1) * D, sizeof v[k]);
    };
    load(first);
    float m = fmaxf(mine[0].x, mine[1].x);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
    const float base = m == -INFINITY ? 0.0f : m;
    float fade[2], l = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      fade[k] = __builtin_amdgcn_exp2f((mine[k].x - base) * c.cs);
      l += mine[k].y * fade[k];
    }
    l = wave_sum(l);
    float o[kCols] = {};
    for (int k0 = first; k0 < last; k0 += 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float all = __shfl(k0 + k < 64 ? fade[0] : fade[1], (k0 + k) & 63);
        const float by = k0 + k < last ? all : 0.0f;
#pragma unroll
        for (int i = 0; i < kCols; ++i) o[i] += by != 0.0f ? v[k][i] * by : 0.0f;
      }
      if (k0 + 8 < last) load(k0 + 8);
    }
    if constexpr (kJoin > 1) {  // one row a workgroup
#pragma unroll
      for (int i = 0; i < kCols; ++i) sums[wave][lane * kCols + i] = o[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        o[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < kJoin; ++k) o[i] += sums[k][lane * kCols + i];
      }
      __syncthreads();
      if (part > 0) continue;
    }
    const int64_t at = token * c.a.out_token + head * c.a.out_head + lane * kCols;
#pragma unroll
    for (int i = 0; i < kCols; ++i) store1(c.a.out, c.a.type, at + i, l != 0.0f ? o[i] / l : 0.0f);
    if (lane == 0 && c.ml) c.ml[id] = make_float2(m, l);
  }
}

// Softmax weights of 16 keys, summed over the columns of a tile.
template <int D>
__device__ __forceinline__ void add_weights(const KeyRegs<D> &kr, int t, bool odd, bool there, int key, const Column &q,
                                            const QueryOperand<D> &f, float2 ml, float cs, float share,
                                            float limit, float4_t &sum) {
  float4_t p = scores16<D>(kr, t, f);
  float unit = f.unit;
  if (__builtin_expect(odd, 0)) {
    p = scores16<D, true>(kr, t, f);
    unit = odd_unit(f.unit);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool seen = q.live && q.g == 0 && there && key + i <= q.hi && key + i >= q.lo;
    sum[i] += seen ? weight_again(__builtin_fmaf(p[i], unit, -ml.x), cs, limit) * share : 0.0f;
  }
}

// Sums of two steps' halves over the 16 columns: lane 16 j + t (t 0 or 1) gets
// those of the four keys of its j of half t.
__device__ __forceinline__ float4_t fold_weights(float4_t v0, float4_t v1) {
  const bool odd = threadIdx.x & 1;
  float4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the even lanes gather half 0, the odd ones half 1
    const float keep = odd ? v1[i] : v0[i], give = odd ? v0[i] : v1[i];
    v[i] = keep + dpp_row_f<kDppQuadXor1>(give);
    v[i] += dpp_row_f<kDppQuadXor2>(v[i]);
    v[i] += dpp_row_f<kDppRowRor4>(v[i]);
    v[i] += dpp_row_f<kDppRowRor8>(v[i]);
  }
  return v;
}

// weights_out += v for four keys from `key` on, those that a query sees: the
// last query at least, and the first one's window.
__device__ __forceinline__ void store_weights(const Call &c, float4_t v, uint64_t at, int key, int64_t len,
                                              int64_t start) {
  const int64_t lo = c.a.window ? start - c.a.window : -1;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (key + i < len && key + i > lo) add_weight(c.a.weights_out + at + i, v[i]);
}

// The weights of the rows of the cache where no sequence's key head has more
// rows than a tile, from the scores again and each query's maximum and sum.  A
// wave takes kWeightSteps steps of a sequence's key head and adds each key's sum
// once; the next step's keys are on their way while this one's are used.  Bound
// by bytes in long contexts, in short ones by the three loads that follow each
// other: 16 sequences of up to 4096 rows, 8 key heads of 128 columns, 17 us (36 MB
// of keys); one step at a time 26 us.  (A store in place of the addition is 15.5,
// but sequences that share a page would lose sums.)
constexpr int kWeightSteps = 8;

template <int D, bool kSmallPages>
__global__ __launch_bounds__(kTileThreads, 2) void kv_weights_kernel(Call c, int parts, int64_t work) {
  constexpr int kChunk = kWeightSteps * kStepKeys;
  const int lane = threadIdx.x & 63, j = lane >> 4, H = c.kv.p.kv_heads;
  const int64_t waves = (int64_t)gridDim.x * kTileWaves;
  for (int64_t item = (int64_t)blockIdx.x * kTileWaves + uniform(threadIdx.x >> 6); item < work; item += waves) {
    const int h = (int)(item / parts % H), s = (int)(item / parts / H);
    const SeqSpan span = seq_span(c.rows, s);
    const int64_t len = c.rows.lengths[s], start = len - span.n;
    const int64_t end = min(len, (int64_t)c.rows.table_width << c.kv.shift);
    if (span.n == 0) continue;
    // a table may be far wider than its sequence: the parts go on to the sequence's end
    for (int64_t key_at = item % parts * kChunk; key_at < end; key_at += (int64_t)parts * kChunk) {
      const int key0 = (int)key_at;
      // queries that see any of these keys
      const int64_t i0 = max((int64_t)key0 - start, (int64_t)0);
      const int64_t i1 = c.a.window ? min(key0 + kChunk - 1 + (int64_t)c.a.window - start, (int64_t)span.n)
                                    : (int64_t)span.n;
      if (i0 >= i1) continue;
      const int32_t *table = c.rows.table + s * c.rows.table_stride;
      const int count = (int)min((end - key0 + kStepKeys - 1) / kStepKeys, (int64_t)kWeightSteps);
      // entries of all steps, a step a lane
      const Entries<kSmallPages> all = entries_of<kSmallPages>(c, table, key0 + min(lane, count - 1) * kStepKeys);
      const int t = lane & 1;  // the half whose weights this lane would store
      const bool mine = (lane & 15) < 2;
      struct Ahead {
        KeyRegs<D> kr;
        uint64_t at;
        bool ok[2];
      } now, next;
      auto load = [&](int n, Ahead &x) {
        Entries<kSmallPages> e;
#pragma unroll
        for (int u = 0; u < (kSmallPages ? 2 : 1); ++u) e.entry[u] = __builtin_amdgcn_readlane(all.entry[u], n);
        const Place<kSmallPages> p = place_of<D>(c, e, h, key0 + n * kStepKeys);
        load_keys<D>(c, p, (lane & 15) / Tile<D>::kRows, x.kr);
        x.at = p.row[kSmallPages ? t : 0] + (kSmallPages ? 0 : 16 * t) + 4 * j;
        x.ok[0] = p.ok[0], x.ok[1] = p.ok[1];
      };
      load(0, now);
      const Column q = column_of<D>(c, span, len, h, 0);
      const float2 ml = q.live ? c.ml[(int64_t)q.token * c.a.q_heads + q.head] : make_float2(0.0f, 0.0f);
      QueryOperand<D> f;
      load_query<D>(c, q, f);
      const float share = share_again(ml.y), limit = limit_again(ml.y);
      for (int n = 0; n < count; ++n) {
        if (n + 1 < count) load(n + 1, next);
        const int key = key0 + n * kStepKeys + 4 * j;
        float4_t sum[2] = {};
        const bool odd = keys_odd<D>(now.kr);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          add_weights<D>(now.kr, u, odd, now.ok[u], key + 16 * u, q, f, ml, c.cs, share, limit, sum[u]);
        const float4_t v = fold_weights(sum[0], sum[1]);
        if (mine && (t ? now.ok[1] : now.ok[0])) store_weights(c, v, now.at, key + 16 * t, len, start);
        now = next;
      }
    }
  }
}

// How the work is split, and where the workspace's parts are.
struct Plan {
  int tiles, tile_waves, few_rows, waves, splits, prompt_splits;
  bool prompts;
  size_t part_o, part_ml, ml, q_halves, q_info, bytes;
};

// Workgroups of tiles that fill the chip: four a CU.  (768: one long sequence 48
// instead of 43 us.)
constexpr int64_t kFill = 1024;
constexpr int64_t kMaxParts = 1ll << 26;  // floats of partial results
// Rows of a sequence's key head that the tiles take; more go to the prompts'
// kernel, whose 256 rows share each expanded key.  (8 sequences of 6000 rows, 8
// key heads of 8 query heads: 64 rows 57 us by the tiles, 72 rows 87 by the
// other; tiles read the keys once for every 32 rows.)
constexpr int kFewRows = 64;
constexpr int64_t kCus = 256;
constexpr int64_t kShortContext = 768, kShortOfMany = 4096;

// On the host, where min and max of HIP's headers are those of int.
int64_t least_of(int64_t a, int64_t b) { return a < b ? a : b; }
int64_t most_of(int64_t a, int64_t b) { return a > b ? a : b; }

// Whether the rows of a sequence's key head are one tile at most, for all that
// the call's sizes tell.
bool one_tile(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, int64_t group) {
  return (r.offsets ? r.tokens : 1) * group <= 16 / (kv.head_dim / kKvGroup);
}

Plan plan_of(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_attention_t &a) {
  Plan p;
  const int64_t group = a.q_heads / kv.kv_heads;
  const int tile_rows = 16 / (kv.head_dim / kKvGroup);
  const int64_t most = (r.offsets ? r.tokens : 1) * group;  // rows that a sequence's key head can have
  // sequences of more rows take the prompts' kernel, if there can be any
  p.prompts = r.offsets && most > kFewRows;
  p.few_rows = p.prompts ? kFewRows : 1 << 30;
  const int tiles = (int)((least_of(most, p.few_rows) + tile_rows - 1) / tile_rows);
  p.tile_waves = tiles >= 4 ? 4 : tiles >= 2 ? 2 : 1;
  p.tiles = (tiles + p.tile_waves - 1) / p.tile_waves * p.tile_waves;
  // keys that a sequence's rows can see
  const int64_t cap = least_of((int64_t)r.table_width * kv.page_size,
                               a.window ? (int64_t)a.window + (r.offsets ? r.tokens : 1) : (int64_t)1 << 30);
  const int64_t out = (int64_t)r.tokens * a.q_heads * kv.head_dim;
  const int64_t parts = most_of(least_of(kMaxParts / most_of(out, 1), 128), 1);
  // workgroups without splits: every sequence's rows, to the tile, need at most this many
  const int64_t groups = (least_of(r.tokens * group, (int64_t)r.seqs * p.few_rows) / (tile_rows * p.tile_waves) + r.seqs) *
                         kv.kv_heads;
  p.splits = (int)most_of(least_of(least_of((kFill + groups - 1) / groups, (cap + 255) / 256), parts), 1);
  // Short contexts: one workgroup of more waves is sooner done than splits and
  // their joining (one sequence of 8 key heads, 64 of queries, 512 keys: 13.4
  // against 14.7 us, 1024: 16.0 against 14.7), for longer where sequences alone
  // give every CU one (32 sequences, 2000 keys: 23.5 against 27.9 us, 4000:
  // 33.4 against 34.8).
  p.waves = 4;
  if (p.splits > 1 && cap <= ((int64_t)r.seqs * kv.kv_heads >= kCus ? kShortOfMany : kShortContext)) {
    p.waves = 8;
    p.splits = 1;
  }
  // the prompts' kernel has at most two workgroups a CU and a join of its own, so three for every CU at most
  p.prompt_splits = 1;
  if (p.prompts) {
    const int64_t blocks = (r.tokens * group / prompt_rows(kv.head_dim) + r.seqs) * kv.kv_heads;
    p.prompt_splits = (int)most_of(least_of(least_of(768 / blocks, (cap + 511) / 512), parts), 1);
  }
  const int64_t rows = (int64_t)r.tokens * a.q_heads;
  const int splits = max(p.splits, p.prompt_splits);
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  size_t at = 0;
  p.part_o = at;
  if (splits > 1) at += up(rows * splits * kv.head_dim * sizeof(float));
  p.part_ml = at;
  if (splits > 1) at += up(rows * splits * sizeof(float2));
  p.ml = at;
  if (a.weights_out) at += up(rows * sizeof(float2));
  // queries for the weights: a tile may read up to 32 rows past the last
  p.q_halves = at;
  const bool halves = a.weights_out && !one_tile(kv, r, group);
  if (halves) at += up((rows + 32) * kv.head_dim * sizeof(_Float16));
  p.q_info = at;
  if (halves) at += up((rows + 32) * sizeof(float4));
  p.bytes = at > 0 ? at : 256;
  return p;
}

unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20); }

template <int D, bool kSmallPages>
hipError_t launch_all(Call &c, hipStream_t s) {
  const int64_t work = (int64_t)c.rows.seqs * c.kv.p.kv_heads * c.splits * (c.tiles / c.tile_waves);
  const bool twice = c.a.type == COLI_MOE_F16;
  const auto kernel = c.waves == 8 ? twice ? kv_attention_kernel<D, true, kSmallPages, 8>
                                           : kv_attention_kernel<D, false, kSmallPages, 8>
                      : twice      ? kv_attention_kernel<D, true, kSmallPages, 4>
                                   : kv_attention_kernel<D, false, kSmallPages, 4>;
  c.blocks = (int)grid_of(work);
  const int64_t copies = (int64_t)c.rows.seqs * c.kv.p.kv_heads * c.copy_parts;
  hipError_t e = launch(kernel, dim3(c.blocks + grid_of(copies)), dim3(64 * c.waves), 0, s, c, work);
  const bool prompts = c.few_rows < 1 << 30;
  if (e == hipSuccess && prompts) e = launch_attention_prompts(c, s);
  if (e == hipSuccess && c.part_splits > 1) {
    // rows of sequences of few rows alone, or of all tokens
    const int64_t few = prompts ? least_of((int64_t)c.rows.tokens * c.group, c.few_rows)
                                : (c.rows.offsets ? (int64_t)c.rows.tokens : 1) * c.group;
    const int64_t by_seq = few * c.rows.seqs * c.kv.p.kv_heads, by_token = (int64_t)c.rows.tokens * c.a.q_heads;
    const bool seqs = c.prompt_splits == 1 && by_seq <= by_token;
    const int64_t rows = seqs ? by_seq : by_token;
    const bool wide = rows <= 1024 && c.part_splits >= 32;
    e = launch(wide ? kv_attention_join_kernel<D, kTileWaves> : kv_attention_join_kernel<D, 1>,
               dim3(grid_of(wide ? rows : (rows + kTileWaves - 1) / kTileWaves)), dim3(kTileThreads), 0, s, c,
               seqs ? (int)few : 0, rows);
  }
  if (e != hipSuccess || !c.a.weights_out) return e;
  const int64_t cap = (int64_t)c.rows.table_width << c.kv.shift, heads = (int64_t)c.rows.seqs * c.kv.p.kv_heads;
  if (!one_tile(c.kv.p, c.rows, c.group)) return launch_row_weights(c, s);
  // four waves a SIMD, or what the table has room for
  const int64_t chunk = kWeightSteps * kStepKeys;
  const int64_t parts = least_of((cap + chunk - 1) / chunk, (4096 + heads - 1) / heads);
  return launch(kv_weights_kernel<D, kSmallPages>, dim3(grid_of((heads * parts + kTileWaves - 1) / kTileWaves)),
                dim3(kTileThreads), 0, s, c, (int)parts, heads * parts);
}

template <int D>
hipError_t launch_all(Call &c, hipStream_t s) {
  return c.kv.p.page_size < kStepKeys ? launch_all<D, true>(c, s) : launch_all<D, false>(c, s);
}

}  // namespace

size_t kv_attention_workspace_bytes(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r,
                                    const coli_moe_kv_attention_t &a) {
  return plan_of(kv, r, a).bytes;
}

hipError_t launch_kv_attention(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_attention_t &a,
                               void *workspace, hipStream_t s) {
  const Plan p = plan_of(kv, r, a);
  char *ws = static_cast<char *>(workspace);
  const float cs = a.scale != 0.0f ? fminf(fmaxf(fabsf(a.scale) * kLog2e, 0x1p-126f), 0x1p127f) : 1.0f;
  Call c{kv_view(kv), r, a, cs, a.q_heads / kv.kv_heads, p.tiles, p.tile_waves, p.few_rows, p.waves, p.splits, p.prompt_splits,
         max(p.splits, p.prompt_splits), reinterpret_cast<float *>(ws + p.part_o), reinterpret_cast<float2 *>(ws + p.part_ml),
         a.weights_out ? reinterpret_cast<float2 *>(ws + p.ml) : nullptr, ws + p.q_halves,
         reinterpret_cast<float4 *>(ws + p.q_info), 0, 0};
  if (a.weights_out && a.weights_out != kv.weights) {
    // as many parts of a sequence's key head as its table has room for, up to four workgroups a CU
    const int64_t heads = (int64_t)r.seqs * kv.kv_heads, chunk = 4 * 64 * p.waves;
    c.copy_parts = (int)least_of(((int64_t)r.table_width * kv.page_size + chunk - 1) / chunk, (kFill + heads - 1) / heads);
  }
  switch (kv.head_dim) {
    case 64: return launch_all<64>(c, s);
    case 128: return launch_all<128>(c, s);
    default: return launch_all<256>(c, s);
  }
}

}  // namespace coli
