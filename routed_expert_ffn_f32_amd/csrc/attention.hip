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
#include "attention.h"

namespace coli {
namespace {

template <int D>
struct Tile {
  static constexpr int kGroups = D / kKvGroup;
  static constexpr int kRows = 16 / kGroups;         // query rows of a tile
  static constexpr int kSteps = D / 32;              // matrix instructions of a score
  static constexpr int kParts = D / 16;              // of a value
  static constexpr int kKeys = D == 256 ? 32 : 64;   // keys of one step of a wave
  static constexpr int kSubs = kKeys / 16;
  static constexpr int kWords = D == 256 ? 2 : 1;    // 16 values' dwords a lane holds of a key
};

__device__ __forceinline__ float max_over_j(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_over_j(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
// Sum over the groups of a row: every lane of the row's columns gets it.
template <int D>
__device__ __forceinline__ float sum_groups(float v) {
  if constexpr (D >= 128) v += dpp_f<kDppRowRor8>(v);
  if constexpr (D >= 256) v += dpp_f<kDppRowRor4>(v);
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
// per row (elements below 2^-28 of the row's largest are rounded).
template <int D>
struct QueryOperand {
  half8_t b[Tile<D>::kSteps];
  float scale;  // of a summed score, with log2 e
};

template <int D>
__device__ __forceinline__ void load_query(const Call &c, const Column &q, QueryOperand<D> &f) {
  constexpr int kSteps = Tile<D>::kSteps;
  const int j = (threadIdx.x >> 4) & 3;
  Raw8 raw[kSteps];
  float top = 0.0f;
  const int64_t base = q.token * c.a.q_token + q.head * c.a.q_head;
#pragma unroll
  for (int w = 0; w < kSteps; ++w) {
    // columns of dword w of this lane: D = 64 has two a lane, D = 256 two sets of four
    const int col = D == 64 ? 16 * j + 8 * w : D == 128 ? 32 * j + 8 * w : 128 * (w / 4) + 32 * j + 8 * (w % 4);
    raw[w].lo = u32x4{0, 0, 0, 0};
    if (q.live && col / kKvGroup == q.g) raw[w] = load_raw8(c.a.q, c.a.type, base + col);
  }
#pragma unroll
  for (int w = 0; w < kSteps; ++w) {
    float v[8];
    unpack8(c.a.type, raw[w], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
  }
  top = max_over_j(top);
  if constexpr (D >= 128) top = fmaxf(top, dpp_f<kDppRowRor8>(top));
  if constexpr (D >= 256) top = fmaxf(top, dpp_f<kDppRowRor4>(top));
  const int ex = lift_exponent(top);
  const float up = lift(ex);
#pragma unroll
  for (int w = 0; w < kSteps; ++w) {
    float v[8];
    unpack8(c.a.type, raw[w], v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f.b[w][2 * e] = (_Float16)(v[e] * up);
      f.b[w][2 * e + 1] = (_Float16)(v[e + 4] * up);
    }
  }
  f.scale = c.a.scale * kLog2e * unlift(ex);
}

// Four neighbouring scales of a column's group.
__device__ __forceinline__ float4_t scales4(uint2 v) {
  return float4_t{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                  __uint_as_float(v.y & 0xFFFF0000u)};
}

// Keys of one step as they stand in memory.
template <int D>
struct KeyRegs {
  u32x4 k[Tile<D>::kSubs][D == 256 ? 2 : 1];
  uint2 s[Tile<D>::kSubs];
};

template <int D>
__device__ __forceinline__ void load_keys(const Call &c, const SubPlace &p, int t, int g, KeyRegs<D> &r) {
  const int lane = threadIdx.x & 63, j = lane >> 4;
  const int ps = c.kv.p.page_size;
  const uint8_t *base = c.kv.p.k_codes + (p.ph * ps + p.slot) * (D / 2);
  const int row = (lane & 15) * (D / 2);
  if constexpr (D == 64) {
    const uint2 v = *reinterpret_cast<const uint2 *>(base + row + 8 * j);
    r.k[t][0] = u32x4{v.x, v.y, 0, 0};
  } else {
#pragma unroll
    for (int w = 0; w < D / 128; ++w)
      r.k[t][w] = *reinterpret_cast<const u32x4 *>(base + row + 64 * w + 16 * j);
  }
  const uint16_t *sc = c.kv.p.k_scales + (p.ph * Tile<D>::kGroups + g) * ps + p.slot + 4 * j;
  r.s[t] = *reinterpret_cast<const uint2 *>(sc);
}

// Scores (times log2 e) of 16 keys: lane (column, j) gets keys 4 j .. 4 j + 3.
template <int D>
__device__ __forceinline__ float4_t scores16(const KeyRegs<D> &r, int t, const QueryOperand<D> &f) {
  float4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < Tile<D>::kSteps; ++w)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_of(r.k[t][w / 4][w % 4]), f.b[w], acc, 0, 0, 0);
  const float4_t sc = scales4(r.s[t]);
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = sum_groups<D>(acc[i] * sc[i]) * f.scale;
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

// One workgroup: `tile_waves` tiles of one sequence's key head over one split
// of their keys; the waves of a tile take its steps of keys in turn and are
// joined in LDS at the end.  kTwice: the weights as the sum of two halves.
template <int D, bool kTwice>
__global__ __launch_bounds__(kTileThreads, 2) void kv_attention_kernel(Call c, int64_t work) {
  using T = Tile<D>;
  constexpr int kOut = T::kRows * D;  // 1024
  __shared__ float so[kTileWaves][kOut];
  __shared__ float2 sml[kTileWaves][T::kRows];
  const int tid = threadIdx.x, lane = tid & 63, j = lane >> 4, wave = uniform(tid >> 6);
  const int H = c.kv.p.kv_heads;
  if (blockIdx.x == 0) clear_outside(c, D);
  for (int64_t item = blockIdx.x; item < work; item += gridDim.x) {
    const int tgroups = c.tiles / c.tile_waves;
    const int tg = (int)(item % tgroups);
    const int64_t rest = item / tgroups;
    const int split = (int)(rest % c.splits), h = (int)(rest / c.splits % H), s = (int)(rest / c.splits / H);
    const SeqSpan span = seq_span(c.rows, s);
    const int rows = span.n * c.group, r0 = tg * c.tile_waves * T::kRows;
    if (r0 >= rows || rows > c.few_rows) continue;
    const int64_t len = c.rows.lengths[s];
    const int32_t *table = c.rows.table + s * c.rows.table_stride;
    const int tile = tg * c.tile_waves + wave % c.tile_waves;
    const int kw = wave / c.tile_waves, kn = kTileWaves / c.tile_waves;
    const int r1 = min(r0 + c.tile_waves * T::kRows, rows) - 1;
    const KeyRange range = keys_of_rows(c, span, len, r0, r1);
    const int64_t begin = range.lo & ~(int64_t)(T::kKeys - 1);
    const int steps = range.hi > range.lo ? (int)((range.hi - begin + T::kKeys - 1) / T::kKeys) : 0;
    const int per = max((steps + c.splits - 1) / c.splits, 4 * kn);  // a split has some work for each wave
    const int s0 = min(split * per, steps), s1 = min(s0 + per, steps);

    const Column q = column_of<D>(c, span, len, h, tile);
    QueryOperand<D> f;
    load_query<D>(c, q, f);
    // rows of this wave's tile alone, for steps that all of them see whole
    const int64_t pmin = len - span.n + min(tile * T::kRows, rows - 1) / c.group;
    const int64_t pmax = len - span.n + min((tile + 1) * T::kRows, rows - 1) / c.group;

    float m = -INFINITY, l = 0.0f, big = 0.0f;  // maximum, sum, largest weight times scale (against m)
    int ex = lift_exponent(0.0f);               // of `big`: the weights are stored times lift(ex)
    float4_t acc[T::kParts];
#pragma unroll
    for (int i = 0; i < T::kParts; ++i) acc[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

    for (int st = s0 + kw; st < s1; st += kn) {
      const int key0 = (int)begin + st * T::kKeys;
      SubPlace place[T::kSubs];
      bool all = true;
#pragma unroll
      for (int t = 0; t < T::kSubs; ++t) {
        place[t] = sub_place(c, table, h, key0 + 16 * t);
        all = all && place[t].ok;
      }
      KeyRegs<D> kr;
#pragma unroll
      for (int t = 0; t < T::kSubs; ++t) load_keys<D>(c, place[t], t, q.g, kr);
      // values: lane (r, j) holds, of keys 4 j .. 4 j + 3 of each 16, the dword of columns 8 r .. 8 r + 7
      uint32_t vw[T::kSubs][4][T::kWords];
      uint2 vs[T::kSubs];
#pragma unroll
      for (int t = 0; t < T::kSubs; ++t) {
        const int ps = c.kv.p.page_size;
        const uint8_t *base = c.kv.p.v_codes + (place[t].ph * ps + place[t].slot) * (D / 2);
        const int word = D == 64 ? (lane & 15) / 2 * 4 : (lane & 15) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int w = 0; w < T::kWords; ++w)
            vw[t][i][w] = *reinterpret_cast<const uint32_t *>(base + (4 * j + i) * (D / 2) + word + 64 * w);
        vs[t] = *reinterpret_cast<const uint2 *>(c.kv.p.v_scales + (place[t].ph * T::kGroups + q.g) * ps +
                                                 place[t].slot + 4 * j);
      }

      float4_t p[T::kSubs], sv[T::kSubs];
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < T::kSubs; ++t) {
        p[t] = scores16<D>(kr, t, f);
        sv[t] = scales4(vs[t]);
      }
      const bool whole = all && key0 + T::kKeys - 1 <= pmin && (!c.a.window || key0 > pmax - c.a.window) && key0 >= 0;
      if (!whole) {
#pragma unroll
        for (int t = 0; t < T::kSubs; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 16 * t + 4 * j + i;
            const bool seen = place[t].ok && key <= q.hi && key >= q.lo;
            p[t][i] = seen ? p[t][i] : -INFINITY;
            sv[t][i] = seen ? sv[t][i] : 0.0f;
          }
      }
#pragma unroll
      for (int t = 0; t < T::kSubs; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, p[t][i]);
      const float m1 = fmaxf(m, max_over_j(top));
      const float base = m1 == -INFINITY ? 0.0f : m1;
      const float fade = __builtin_amdgcn_exp2f(m - base);
      float sum = 0.0f, most = 0.0f;
#pragma unroll
      for (int t = 0; t < T::kSubs; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = __builtin_amdgcn_exp2f(p[t][i] - base);
          sum += e;
          p[t][i] = e * sv[t][i];
          most = fmaxf(most, fabsf(p[t][i]));
        }
      m = m1;
      l = l * fade + sum;
      big = fmaxf(big * fade, max_over_j(most));
      const int ex1 = lift_exponent(big);
      const float turn = __builtin_amdgcn_ldexpf(fade, ex - ex1);
      ex = ex1;
      if (__any(turn != 1.0f)) {
#pragma unroll
        for (int i = 0; i < T::kParts; ++i) acc[i] *= turn;
      }
      const float up = lift(ex);
#pragma unroll
      for (int t = 0; t < T::kSubs; t += 2) {
        half8_t b, b2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = p[t + i / 4][i % 4] * up;
          b[i] = (_Float16)v;
          if constexpr (kTwice) b2[i] = (_Float16)(v - (float)b[i]);
        }
        uint32_t v[8][T::kWords];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int w = 0; w < T::kWords; ++w) v[i][w] = vw[t + i / 4][i % 4][w] ^ 0x88888888u;
        // D = 64: a lane's four columns are one half of its dword
        const uint32_t half = D == 64 ? 0x00020002u * (lane & 1) : 0u;
#pragma unroll
        for (int i = 0; i < T::kParts; i += 2) {
          const uint32_t sel = (0x0C040C00u + 0x00010001u * (i / 2 % 4)) + half;
          u32x4 lo, hi;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t two = __builtin_amdgcn_perm(v[2 * e + 1][i / 8], v[2 * e][i / 8], sel);
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
      }
    }

    // this wave's sums, against its maximum: to LDS
    l = sum_over_j(l);
    const float down = unlift(ex);
    const int col = lane & 15, r = col % T::kRows;
    __syncthreads();  // of the item before, all is read
    if (j == 0 && q.g == 0) sml[wave][r] = make_float2(m, l);
#pragma unroll
    for (int i = 0; i < T::kParts; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = D == 64 ? 16 * j + 4 * e + i : 128 * (i / 8) + 32 * j + 8 * e + i % 8;
        if (d / kKvGroup == q.g) so[wave][r * D + d] = acc[i][e] * down;
      }
    __syncthreads();
    for (int e = tid; e < c.tile_waves * kOut; e += kTileThreads) {
      const int tw = e / kOut, rr = e % kOut / D, d = e % D;
      const int row = r0 + tw * T::kRows + rr;
      if (row >= rows) continue;
      float mm = -INFINITY;
      for (int k = 0; k < kn; ++k) mm = fmaxf(mm, sml[k * c.tile_waves + tw][rr].x);
      const float base = mm == -INFINITY ? 0.0f : mm;
      float o = 0.0f, ll = 0.0f;
      for (int k = 0; k < kn; ++k) {
        const int w = k * c.tile_waves + tw;
        const float2 v = sml[w][rr];
        const float fade = __builtin_amdgcn_exp2f(v.x - base);
        ll += v.y * fade;
        o += so[w][rr * D + d] * fade;
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

// Joins the splits of a row: one wave a row, D / 64 columns a lane.
template <int D>
__global__ __launch_bounds__(kTileThreads) void kv_attention_join_kernel(Call c) {
  constexpr int kCols = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * kTileWaves, n = (int64_t)c.rows.tokens * c.a.q_heads;
  for (int64_t id = (int64_t)blockIdx.x * kTileWaves + uniform(threadIdx.x >> 6); id < n; id += waves) {
    const int token = (int)(id / c.a.q_heads), head = (int)(id % c.a.q_heads);
    const int s = find_seq(c.rows, token);
    if (s < 0) continue;
    const int splits = seq_span(c.rows, s).n * c.group <= c.few_rows ? c.splits : c.prompt_splits;
    if (splits == 1) continue;
    const float2 *ml = c.part_ml + id * c.part_splits;
    float m = -INFINITY;
    for (int k = 0; k < splits; ++k) m = fmaxf(m, ml[k].x);
    const float base = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, o[kCols] = {};
    for (int k = 0; k < splits; ++k) {
      const float fade = __builtin_amdgcn_exp2f(ml[k].x - base);
      l += ml[k].y * fade;
#pragma unroll
      for (int i = 0; i < kCols; ++i) o[i] += c.part_o[(id * c.part_splits + k) * D + lane * kCols + i] * fade;
    }
    const int64_t at = token * c.a.out_token + head * c.a.out_head + lane * kCols;
#pragma unroll
    for (int i = 0; i < kCols; ++i) store1(c.a.out, c.a.type, at + i, l != 0.0f ? o[i] / l : 0.0f);
    if (lane == 0 && c.ml) c.ml[id] = make_float2(m, l);
  }
}

// weights_out = weights + sums of the softmax weights of each row of the
// cache, from the scores again and each query's maximum and sum.  A wave
// takes one step of keys of a sequence's key head and all tiles of queries
// that see any of them, so that a place has one writer.
template <int D>
__global__ __launch_bounds__(kTileThreads, 2) void kv_weights_kernel(Call c, int chunks, int64_t work) {
  using T = Tile<D>;
  const int lane = threadIdx.x & 63, j = lane >> 4, H = c.kv.p.kv_heads;
  const int64_t waves = (int64_t)gridDim.x * kTileWaves;
  for (int64_t item = (int64_t)blockIdx.x * kTileWaves + uniform(threadIdx.x >> 6); item < work; item += waves) {
    const int key0 = (int)(item % chunks) * T::kKeys;
    const int h = (int)(item / chunks % H), s = (int)(item / chunks / H);
    const SeqSpan span = seq_span(c.rows, s);
    const int64_t len = c.rows.lengths[s], start = len - span.n;
    if (span.n == 0 || key0 >= len) continue;
    // queries that see any of the step's keys
    const int64_t i0 = max((int64_t)key0 - start, (int64_t)0);
    const int64_t i1 = c.a.window ? min(key0 + T::kKeys - 1 + (int64_t)c.a.window - start, (int64_t)span.n)
                                  : (int64_t)span.n;
    if (i0 >= i1) continue;
    const int32_t *table = c.rows.table + s * c.rows.table_stride;
    SubPlace place[T::kSubs];
    KeyRegs<D> kr;
    const int g = (lane & 15) / T::kRows;
#pragma unroll
    for (int t = 0; t < T::kSubs; ++t) {
      place[t] = sub_place(c, table, h, key0 + 16 * t);
      load_keys<D>(c, place[t], t, g, kr);
    }
    float4_t sum[T::kSubs];
#pragma unroll
    for (int t = 0; t < T::kSubs; ++t) sum[t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const int last = (int)((i1 * c.group - 1) / T::kRows);
    for (int tile = (int)(i0 * c.group / T::kRows); tile <= last; ++tile) {
      const Column q = column_of<D>(c, span, len, h, tile);
      QueryOperand<D> f;
      load_query<D>(c, q, f);
      const float2 ml = q.live ? c.ml[(int64_t)q.token * c.a.q_heads + q.head] : make_float2(0.0f, 0.0f);
      const float share = ml.y != 0.0f ? 1.0f / ml.y : 0.0f;
#pragma unroll
      for (int t = 0; t < T::kSubs; ++t) {
        const float4_t p = scores16<D>(kr, t, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key0 + 16 * t + 4 * j + i;
          const bool seen = q.live && q.g == 0 && place[t].ok && key <= q.hi && key >= q.lo;
          sum[t][i] += seen ? __builtin_amdgcn_exp2f(p[i] - ml.x) * share : 0.0f;
        }
      }
    }
    // over the 16 columns: one lane of each j stores its four keys
#pragma unroll
    for (int t = 0; t < T::kSubs; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = sum[t][i];
        v += dpp_f<kDppQuadXor1>(v);
        v += dpp_f<kDppQuadXor2>(v);
        v += dpp_f<kDppRowRor4>(v);
        v += dpp_f<kDppRowRor8>(v);
        sum[t][i] = v;
      }
      if ((lane & 15) != t || !place[t].ok) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t key = key0 + 16 * t + 4 * j + i;
        // seen by the last query at least, and by the first one's window
        if (key >= len || (c.a.window && key <= start - c.a.window)) continue;
        const int64_t at = place[t].ph * c.kv.p.page_size + place[t].slot + 4 * j + i;
        c.a.weights_out[at] = c.kv.p.weights[at] + sum[t][i];
      }
    }
  }
}

// How the work is split, and where the workspace's parts are.
struct Plan {
  int tiles, tile_waves, few_rows, splits, prompt_splits;
  bool prompts;
  size_t part_o, part_ml, ml, bytes;
};

constexpr int64_t kFill = 1024;             // workgroups of tiles that fill the chip (four a CU)
constexpr int64_t kMaxParts = 1ll << 26;    // floats of partial results
constexpr int kFewRows = 64;

Plan plan_of(const coli_moe_kv_t &kv, const coli_moe_kv_rows_t &r, const coli_moe_kv_attention_t &a) {
  Plan p;
  const int64_t group = a.q_heads / kv.kv_heads;
  const int tile_rows = 16 / (kv.head_dim / kKvGroup);
  const int64_t most = (r.offsets ? r.tokens : 1) * group;  // rows that a sequence's key head can have
  // sequences of more rows take the prompts' kernel, if there can be any
  p.prompts = r.offsets && most > kFewRows;
  p.few_rows = p.prompts ? kFewRows : 1 << 30;
  const int tiles = (int)((min(most, (int64_t)p.few_rows) + tile_rows - 1) / tile_rows);
  p.tile_waves = tiles >= 4 ? 4 : tiles >= 2 ? 2 : 1;
  p.tiles = (tiles + p.tile_waves - 1) / p.tile_waves * p.tile_waves;
  const int64_t cap = (int64_t)r.table_width * kv.page_size;
  const int64_t out = (int64_t)r.tokens * a.q_heads * kv.head_dim;
  const int64_t parts = max(min(kMaxParts / max(out, (int64_t)1), (int64_t)128), (int64_t)1);
  // workgroups without splits: every sequence's rows, to the tile, need at most this many
  const int64_t groups = (min(r.tokens * group, (int64_t)r.seqs * p.few_rows) / (tile_rows * p.tile_waves) + r.seqs) *
                         kv.kv_heads;
  p.splits = (int)max(min(min((kFill + groups - 1) / groups, (cap + 255) / 256), parts), (int64_t)1);
  p.prompt_splits = 1;
  if (p.prompts) {
    const int64_t blocks = (r.tokens * group / prompt_rows(kv.head_dim) + r.seqs) * kv.kv_heads;
    p.prompt_splits = (int)max(min(min(1536 / blocks, (cap + 511) / 512), parts), (int64_t)1);
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
  p.bytes = at > 0 ? at : 256;
  return p;
}

unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20); }

template <int D>
hipError_t launch_all(const Call &c, hipStream_t s) {
  const int64_t work = (int64_t)c.rows.seqs * c.kv.p.kv_heads * c.splits * (c.tiles / c.tile_waves);
  const auto kernel = c.a.type == COLI_MOE_F16 ? kv_attention_kernel<D, true> : kv_attention_kernel<D, false>;
  hipError_t e = launch(kernel, dim3(grid_of(work)), dim3(kTileThreads), 0, s, c, work);
  if (e == hipSuccess && c.few_rows < 1 << 30) e = launch_attention_prompts(c, s);
  if (e == hipSuccess && c.part_splits > 1) {
    const int64_t blocks = ((int64_t)c.rows.tokens * c.a.q_heads + kTileWaves - 1) / kTileWaves;
    e = launch(kv_attention_join_kernel<D>, dim3(grid_of(blocks)), dim3(kTileThreads), 0, s, c);
  }
  if (e == hipSuccess && c.a.weights_out) {
    const int64_t cap = (int64_t)c.rows.table_width << c.kv.shift;
    const int chunks = (int)((cap + Tile<D>::kKeys - 1) / Tile<D>::kKeys);
    const int64_t items = (int64_t)c.rows.seqs * c.kv.p.kv_heads * chunks;
    e = launch(kv_weights_kernel<D>, dim3(grid_of((items + kTileWaves - 1) / kTileWaves)), dim3(kTileThreads), 0, s, c,
               chunks, items);
  }
  return e;
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
  Call c{kv_view(kv), r, a, a.q_heads / kv.kv_heads, p.tiles, p.tile_waves, p.few_rows, p.splits, p.prompt_splits,
         max(p.splits, p.prompt_splits), reinterpret_cast<float *>(ws + p.part_o), reinterpret_cast<float2 *>(ws + p.part_ml),
         a.weights_out ? reinterpret_cast<float2 *>(ws + p.ml) : nullptr};
  switch (kv.head_dim) {
    case 64: return launch_all<64>(c, s);
    case 128: return launch_all<128>(c, s);
    default: return launch_all<256>(c, s);
  }
}

}  // namespace coli
