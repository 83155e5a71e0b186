// Attention over the paged 4-bit cache for sequences with many query rows
// (tokens times query heads of a key head): prompts.
//
// A workgroup takes 256 rows of one sequence's key head, 32 a wave.  Steps of
// keys are expanded once for all of them, into LDS as halves: K' [key][column]
// and V' [column][key], and both products are 32x32x16 matrix instructions,
// transposed, S = K' Q^T and O = V'^T P^T, so that the weights P come out of
// the first in the layout that the second wants (keys in the order 0-3, 8-11,
// 4-7, 12-15 of every 16) and each lane has one query: its maximum, sum and
// rescaling are a lane's own numbers.  While a step is computed the codes of
// the next one are on their way from memory.
//
// A code times its scale, 4 and 8 significant bits, is exact in a half; what
// the exponent lacks is made up by one power of two for the keys and one for
// the values of each step.  Where the scales of a step's values are more than
// 25 powers of two apart, the small ones follow in passes of their own, so a
// value counts down to 2^-77 of the largest next to it.  Rows whose scale is
// NaN (or Inf) stay out of the products, where 0 times NaN would reach rows
// that do not see them, and are put on those that do.
//
// Bound: 4 D flops of the matrix cores a score against about 9 vector
// instructions, one of them an exponential at a quarter of the rate, and 2
// more for the expansion, shared by 256 rows: the vector units are the busier.
#include "attention.h"

namespace coli {
namespace {

typedef float float16_t __attribute__((ext_vector_type(16)));

constexpr int kBand = 26;    // powers of two of one pass over the values
constexpr int kBands = 3;
constexpr int kMayCross = 0x16;  // what the scheduler may move between groups of matrix instructions: vector, scalar, global
constexpr float kSlack = 8;  // the maximum may be passed by 2^8 before sums are rescaled

template <int D>
struct Prompt {
  static constexpr int kRows = prompt_rows(D);      // of a workgroup, 32 a wave
  static constexpr int kThreads = 2 * kRows;
  static constexpr int kWaves = kThreads / 64;
  static constexpr int kGroups = D / kKvGroup;
  static constexpr int kKeys = D == 256 ? 32 : 64;  // of a step
  static constexpr int kSubs = kKeys / 32;
  static constexpr int kSteps = D / 16;   // instructions of 32 keys' scores
  static constexpr int kParts = D / 32;   // pieces of 32 columns of a result
  // K' [key][column] and V' [column][key] in halves.  16 bytes more than a row
  // move neighbouring rows to other banks, for 16-byte reads of 16 rows at a
  // time.  Column 8 o + b of V' is row b D / 8 + o, so that the rows that
  // neighbouring lanes write are neighbours too, and a lane ends up with 8
  // columns of a result side by side.
  static constexpr int kKeyRow = D + 8, kValRow = kKeys + 8;
  static constexpr int kOct = D / 8;
  // One thread's unit of a step's expansion: 4 keys' values of 8 columns (half
  // of the waves), or one key's 32 columns (D = 64: 16).
  static constexpr int kPieces = D == 64 ? 4 : D / 32;
  static constexpr int kStagers = kThreads / 2;
  static constexpr int kUnits = kKeys * kPieces / kStagers;  // of a thread
  static constexpr int kUnitKeys = kStagers / kPieces;       // keys from one unit to the next
  static_assert(kUnits >= 1 && kUnitKeys * kUnits == kKeys && kUnitKeys % 16 == 0, "units cover a step");
};

__device__ __forceinline__ int wave_max(int v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = max(v, __shfl_xor(v, d));
  return uniform(v);
}

// Exponents of the scales of a step: largest of the keys', largest and
// smallest (of those not 0) of the values', and whether one is NaN or Inf.
struct StepScales {
  int k, v, v_least;
  bool bad;
};

// 2^-(exponent - 11): brings the largest scale to [2^11, 2^12), its values to
// 2^15 at most.
__device__ __forceinline__ int scale_exponent(int e) { return max(e, 12); }
__device__ __forceinline__ float scale_up(int ex) { return __uint_as_float((uint32_t)(265 - ex) << 23); }
__device__ __forceinline__ float scale_unit(int ex) { return __uint_as_float((uint32_t)(ex - 11) << 23); }

// A scale (times up) as a half, 0 for those that stay out: NaN, Inf, and of the
// values those outside the band.
__device__ __forceinline__ _Float16 key_scale(uint32_t bf16, float up) {
  return (_Float16)((bf16 & 0x7F80) == 0x7F80 ? 0.0f : __uint_as_float(bf16 << 16) * up);
}
__device__ __forceinline__ _Float16 val_scale(uint32_t bf16, float up, int limit) {
  const int e = (int)(bf16 >> 7) & 255;
  return (_Float16)(e == 255 || e > limit || e <= limit - kBand ? 0.0f : __uint_as_float(bf16 << 16) * up);
}

__device__ __forceinline__ uint32_t times(uint32_t codes, half2_t s) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, codes) * s);
}

// A unit of the next step as it stands in memory.
struct Staged {
  u32x4 code;
  uint2 scale;
};

template <int D, bool kTwice>
__global__ __launch_bounds__(Prompt<D>::kThreads, D == 256 ? 1 : 2) void kv_prompt_kernel(Call c, int64_t work) {
  using T = Prompt<D>;
  __shared__ __align__(16) _Float16 lk[2][T::kKeys * T::kKeyRow];
  __shared__ __align__(16) _Float16 lv[2][D * T::kValRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), hf = lane >> 5, l32 = lane & 31;
  const int H = c.kv.p.kv_heads, ps = c.kv.p.page_size, S = c.rows.seqs;

  for (int64_t item = blockIdx.x; item < work; item += gridDim.x) {
    const int h = (int)(item % H), split = (int)(item / H % c.prompt_splits);
    // the last tiles of a sequence see the most keys: they come first
    const int64_t tiles = work / H / c.prompt_splits, b = tiles - 1 - item / H / c.prompt_splits;
    // sequence s has the tiles from first_token * group / 256 + s on: room for all of its rows
    int s = 0, n = S;
    while (n > 1) {
      const int step = (n + 63) / 64, i = lane * step;
      const bool below =
          i < n && (int64_t)min(max(c.rows.offsets[s + i], 0), c.rows.tokens) * c.group / T::kRows + s + i <= b;
      const int k = max(__popcll(__ballot(below)), 1);
      s += (k - 1) * step;
      n = min(step, n - (k - 1) * step);
    }
    s = uniform(s);
    const SeqSpan span = seq_span(c.rows, s);
    const int rows = span.n * c.group;
    const int64_t tile = b - ((int64_t)span.first * c.group / T::kRows + s);
    if (rows <= c.few_rows || tile < 0 || tile * T::kRows >= rows) continue;
    const int r0 = (int)tile * T::kRows, r1 = min(r0 + T::kRows, rows) - 1;
    const int64_t len = c.rows.lengths[s];
    const int32_t *table = c.rows.table + s * c.rows.table_stride;
    const KeyRange range = keys_of_rows(c, span, len, r0, r1);
    const int64_t begin = range.lo & ~(int64_t)(T::kKeys - 1);
    const int steps = range.hi > range.lo ? (int)((range.hi - begin + T::kKeys - 1) / T::kKeys) : 0;
    const int per = max((steps + c.prompt_splits - 1) / c.prompt_splits, 2);
    const int s0 = min(split * per, steps), s1 = min(s0 + per, steps);

    // this lane's query
    const int row = r0 + wave * 32 + l32;
    const bool live = row < rows;
    const int qi = live ? row / c.group : 0;
    const int token = span.first + qi, head = h * c.group + (live ? row % c.group : 0);
    const int64_t pos = len - span.n + qi;
    const int q_hi = live ? (int)min(max(pos, (int64_t)-1), (int64_t)1 << 30) : -1;
    const int q_lo = c.a.window ? (int)min(max(pos - c.a.window + 1, (int64_t)0), (int64_t)1 << 30) : 0;
    // and the wave's rows: keys that any and that all of them see
    const int w0 = min(r0 + wave * 32, rows - 1), w1 = min(r0 + wave * 32 + 31, rows - 1);
    const bool any = r0 + wave * 32 < rows;
    const int64_t p0 = len - span.n + w0 / c.group, p1 = len - span.n + w1 / c.group;
    const int64_t any_lo = c.a.window ? p0 - c.a.window + 1 : 0, all_lo = c.a.window ? p1 - c.a.window + 1 : 0;

    half8_t q[T::kSteps];
    float q_scale;
    {
      Raw8 raw[T::kSteps];
      const int64_t base = token * c.a.q_token + head * c.a.q_head;
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < T::kSteps; ++i) {
        raw[i].lo = u32x4{0, 0, 0, 0};
        if (live) raw[i] = load_raw8(c.a.q, c.a.type, base + 16 * i + 8 * hf);
      }
#pragma unroll
      for (int i = 0; i < T::kSteps; ++i) {
        float v[8];
        unpack8(c.a.type, raw[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
      }
      top = fmaxf(top, __shfl_xor(top, 32));
      const int ex = lift_exponent(top);
      // the sign of the scale goes with the query, a scale of 0 makes it 0: what multiplies scores is positive
      const float up = c.a.scale > 0.0f ? lift(ex) : c.a.scale < 0.0f ? -lift(ex) : 0.0f;
#pragma unroll
      for (int i = 0; i < T::kSteps; ++i) {
        float v[8];
        unpack8(c.a.type, raw[i], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q[i][2 * e] = (_Float16)(v[e] * up);
          q[i][2 * e + 1] = (_Float16)(v[e + 4] * up);
        }
      }
      q_scale = c.a.scale != 0.0f ? fabsf(c.a.scale) * kLog2e * unlift(ex) : 1.0f;
    }

    float16_t acc[T::kParts];
#pragma unroll
    for (int i = 0; i < T::kParts; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
    float m = -INFINITY, sum = 0.0f;  // the maximum that the sums stand against; the sum of 2^7 times the weights

    // --- staging ---
    const bool for_values = wave < T::kWaves / 2;
    const int st = tid & (T::kStagers - 1);
    // values: keys 4 quad .. + 3, columns 8 oct .. + 7; keys: key, columns 32 (D = 64: 16) piece ..
    const int oct = st % T::kOct, quad = st / T::kOct;
    const int piece = st % T::kPieces, key = st / T::kPieces;
    const bool stages = !for_values || quad < T::kKeys / 4;
    const int my_key = for_values ? 4 * quad : key;  // of the step, for the first unit
    const int scale_key = lane % T::kKeys;

    auto page_of = [&](int step, int k) {  // of key k of a step, -1 where none or none is seen
      const int64_t at = begin + (int64_t)step * T::kKeys + k;
      return step < s1 && at < range.hi ? row_page(c.kv, table, c.rows.table_width, at) : -1;
    };
    // scales of a step, one key a lane
    uint32_t sk[T::kGroups], sv[T::kGroups];
    auto load_scales = [&](int step, int page) {
      const int slot = ((int)begin + step * T::kKeys + scale_key) & (ps - 1);
      const int64_t at = ((int64_t)max(page, 0) * H + h) * T::kGroups * ps + slot;
#pragma unroll
      for (int g = 0; g < T::kGroups; ++g) {
        sk[g] = c.kv.p.k_scales[at + g * ps];
        sv[g] = c.kv.p.v_scales[at + g * ps];
      }
      const bool there = page >= 0;
#pragma unroll
      for (int g = 0; g < T::kGroups; ++g) {
        sk[g] = there ? sk[g] : 0u;
        sv[g] = there ? sv[g] : 0u;
      }
    };
    auto step_scales = [&]() {
      int k = 0, v = 0, least = 254, bad = 0;
#pragma unroll
      for (int g = 0; g < T::kGroups; ++g) {
        const int ek = (int)(sk[g] >> 7) & 255, ev = (int)(sv[g] >> 7) & 255;
        bad |= ek == 255 || ev == 255;
        k = max(k, ek == 255 ? 0 : ek);
        v = max(v, ev == 255 ? 0 : ev);
        least = min(least, (sv[g] & 0x7FFF) == 0 || ev == 255 ? 254 : ev);
      }
      StepScales r;
      // three 8-bit maxima at a time
      const int packed = wave_max(k | bad << 8);  // bad is the larger digit: the key maximum is taken again if set
      r.bad = packed >> 8;
      r.k = r.bad ? wave_max(k) : packed & 255;
      r.v = wave_max(v);
      r.v_least = 254 - wave_max(254 - least);
      return r;
    };
    auto load_codes = [&](int step, int page, int unit_key, Staged &g) {
      const int slot = ((int)begin + step * T::kKeys + unit_key) & (ps - 1);
      const int64_t ph = (int64_t)max(page, 0) * H + h;
      if (for_values) {
        if (!stages) return;
        const uint8_t *base = c.kv.p.v_codes + (ph * ps + slot) * (D / 2) + 4 * oct;
#pragma unroll
        for (int i = 0; i < 4; ++i) g.code[i] = *reinterpret_cast<const uint32_t *>(base + i * (D / 2));
        g.scale = *reinterpret_cast<const uint2 *>(c.kv.p.v_scales +
                                                   (ph * T::kGroups + 8 * oct / kKvGroup) * ps + slot);
      } else {
        const uint8_t *base = c.kv.p.k_codes + (ph * ps + slot) * (D / 2);
        if constexpr (D == 64) {
          const uint2 v = *reinterpret_cast<const uint2 *>(base + 8 * piece);
          g.code = u32x4{v.x, v.y, 0, 0};
        } else {
          g.code = *reinterpret_cast<const u32x4 *>(base + 16 * piece);
        }
        const int group = piece * (D == 64 ? 16 : 32) / kKvGroup;
        g.scale.x = c.kv.p.k_scales[(ph * T::kGroups + group) * ps + slot];
      }
    };
    // keys of this thread's unit that take part: those before the range's end, on a page
    auto expand_values = [&](int step, int page, int unit_key, const Staged &g, _Float16 *to, int ex, int limit) {
      if (!stages) return;
      const int64_t k0 = begin + (int64_t)step * T::kKeys + unit_key;
      const float up = scale_up(ex);
      half2_t s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t two = i ? g.scale.y : g.scale.x;
        const uint32_t a = page >= 0 && k0 + 2 * i < range.hi ? two & 0xFFFFu : 0u;
        const uint32_t d = page >= 0 && k0 + 2 * i + 1 < range.hi ? two >> 16 : 0u;
        s[i] = half2_t{val_scale(a, up, limit), val_scale(d, up, limit)};
      }
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = g.code[i] ^ 0x88888888u;
      const int chunk = unit_key / 16 * 2 + (quad & 1), half = quad >> 1 & 1;
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint32_t sel = 0x0C040C00u + 0x00010001u * (i / 2);
        const uint32_t t0 = __builtin_amdgcn_perm(w[1], w[0], sel), t1 = __builtin_amdgcn_perm(w[3], w[2], sel);
        const uint2 lo = make_uint2(times(low_codes(t0), s[0]), times(low_codes(t1), s[1]));
        const uint2 hi = make_uint2(times(high_codes(t0), s[0]), times(high_codes(t1), s[1]));
        _Float16 *at = to + (i * T::kOct + oct) * T::kValRow + 8 * chunk + 4 * half;
        *reinterpret_cast<uint2 *>(at) = lo;
        *reinterpret_cast<uint2 *>(at + T::kOct * T::kValRow) = hi;
      }
    };
    auto expand_keys = [&](int step, int page, int unit_key, const Staged &g, _Float16 *to, int ex) {
      const int64_t k0 = begin + (int64_t)step * T::kKeys + unit_key;
      const _Float16 one = key_scale(page >= 0 && k0 < range.hi ? g.scale.x & 0xFFFFu : 0u, scale_up(ex));
      const half2_t s = {one, one};
#pragma unroll
      for (int i = 0; i < (D == 64 ? 2 : 4); ++i) {
        u32x4 v = __builtin_bit_cast(u32x4, codes_of(g.code[i]));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = times(v[e], s);
        *reinterpret_cast<u32x4 *>(to + unit_key * T::kKeyRow + 8 * (piece * (D == 64 ? 2 : 4) + i)) = v;
      }
    };
    // Operands are read four instructions ahead of the four that use them and no
    // further: left alone, the compiler reads so many ahead that registers spill.
    auto product = [&](const _Float16 *from, const half8_t (&p)[T::kKeys / 16], const half8_t (&p2)[T::kKeys / 16]) {
      constexpr int kCount = T::kKeys / 16 * T::kParts;
      half8_t a[2][4];
      auto read = [&](int g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = 4 * g + j, u = n / T::kParts, i = n % T::kParts;
          if (n < kCount)
            a[g & 1][j] = *reinterpret_cast<const half8_t *>(from + (32 * i + l32) * T::kValRow + 8 * (2 * u + hf));
        }
      };
      read(0);
#pragma unroll
      for (int g = 0; g < kCount / 4; ++g) {
        read(g + 1);
        __builtin_amdgcn_sched_barrier(kMayCross);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = 4 * g + j, u = n / T::kParts, i = n % T::kParts;
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[g & 1][j], p[u], acc[i], 0, 0, 0);
          if constexpr (kTwice) acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[g & 1][j], p2[u], acc[i], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(kMayCross);
      }
    };
    auto scores = [&](const _Float16 *from, float16_t (&x)[T::kSubs]) {
      constexpr int kCount = T::kSubs * T::kSteps;
      half8_t a[2][4];
      auto read = [&](int g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = 4 * g + j, i = n / T::kSubs, t = n % T::kSubs;
          if (n < kCount)
            a[g & 1][j] = *reinterpret_cast<const half8_t *>(from + (32 * t + l32) * T::kKeyRow + 8 * (2 * i + hf));
        }
      };
      read(0);
#pragma unroll
      for (int g = 0; g < kCount / 4; ++g) {
        read(g + 1);
        __builtin_amdgcn_sched_barrier(kMayCross);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = 4 * g + j, i = n / T::kSubs, t = n % T::kSubs;
          x[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[g & 1][j], q[i], x[t], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(kMayCross);
      }
    };

    // all units of this thread
    auto pages_of = [&](int step, int (&to)[T::kUnits]) {
#pragma unroll
      for (int u = 0; u < T::kUnits; ++u) to[u] = page_of(step, my_key + u * T::kUnitKeys);
    };
    auto load_units = [&](int step, const int (&pages)[T::kUnits], Staged (&to)[T::kUnits]) {
#pragma unroll
      for (int u = 0; u < T::kUnits; ++u) load_codes(step, pages[u], my_key + u * T::kUnitKeys, to[u]);
    };
    auto expand_units = [&](int step, const int (&pages)[T::kUnits], const Staged (&from)[T::kUnits], int buf, int k_ex,
                            int v_ex) {
#pragma unroll
      for (int u = 0; u < T::kUnits; ++u) {
        const int unit_key = my_key + u * T::kUnitKeys;
        if (for_values)
          expand_values(step, pages[u], unit_key, from[u], lv[buf], v_ex, v_ex);
        else
          expand_keys(step, pages[u], unit_key, from[u], lk[buf], k_ex);
      }
    };

    int unit = 12;  // exponent of the values' power of two that acc stands in
    StepScales now;
    uint64_t there = 0;  // keys of the step that are on a page
    Staged g[T::kUnits];
    int page[T::kUnits], now_page[T::kUnits], scale_page = page_of(s0, scale_key);
    int now_unit = 12;
    pages_of(s0, page);
    __syncthreads();  // of the item before, all is read
    if (s0 < s1) {
      load_scales(s0, scale_page);
      load_units(s0, page, g);
      there = __ballot(scale_page >= 0);
      now = step_scales();
      now_unit = scale_exponent(now.v);
      unit = now_unit;
      expand_units(s0, page, g, 0, scale_exponent(now.k), now_unit);
#pragma unroll
      for (int u = 0; u < T::kUnits; ++u) now_page[u] = page[u];
      pages_of(s0 + 1, page);
      scale_page = page_of(s0 + 1, scale_key);
    }
    __syncthreads();

    for (int step = s0; step < s1; ++step) {
      const int buf = (step - s0) & 1;
      const bool more = step + 1 < s1;
      int page2[T::kUnits], scale_page2 = -1;
      if (more) {
        load_scales(step + 1, scale_page);
        load_units(step + 1, page, g);
        pages_of(step + 2, page2);
        scale_page2 = page_of(step + 2, scale_key);
      }
      const int key0 = (int)begin + step * T::kKeys;
      const bool seen = any && key0 <= p1 && key0 + T::kKeys > any_lo;
      half8_t p[T::kKeys / 16], p2[T::kKeys / 16];
      if (seen) {
        float16_t x[T::kSubs];
#pragma unroll
        for (int t = 0; t < T::kSubs; ++t) {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[t][e] = 0.0f;
        }
        scores(lk[buf], x);
        const bool whole = key0 + T::kKeys - 1 <= p0 && key0 >= all_lo && there == ~0ull;
        if (!whole) {
          const uint64_t mine = there >> (4 * hf);
#pragma unroll
          for (int t = 0; t < T::kSubs; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int at = 32 * t + 8 * (e / 4) + e % 4, k = key0 + at + 4 * hf;
              x[t][e] = k <= q_hi && k >= q_lo && (mine >> at & 1) ? x[t][e] : -INFINITY;
            }
        }
        const float f = q_scale * scale_unit(scale_exponent(now.k));
        float top = x[0][0];
#pragma unroll
        for (int t = 0; t < T::kSubs; ++t)
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, x[t][e]);
        top = fmaxf(top, __shfl_xor(top, 32)) * f;
        if (__any(top > m + kSlack)) {
          const float m1 = fmaxf(m, top);
          const float fade = __builtin_amdgcn_exp2f(m - (m1 == -INFINITY ? 0.0f : m1));
          m = m1;
          sum *= fade;
#pragma unroll
          for (int i = 0; i < T::kParts; ++i) acc[i] *= fade;
        }
        const float base = (m == -INFINITY ? 0.0f : m) - 7.0f;
#pragma unroll
        for (int t = 0; t < T::kSubs; ++t)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float v = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][e], f, -base));
            sum += v;
            const _Float16 hi = (_Float16)v;
            p[2 * t + e / 8][e % 8] = hi;
            if constexpr (kTwice) p2[2 * t + e / 8][e % 8] = (_Float16)(v - (float)hi);
          }
        if (unit != now_unit) {
#pragma unroll
          for (int i = 0; i < T::kParts; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][e] = __builtin_amdgcn_ldexpf(acc[i][e], unit - now_unit);
        }
        product(lv[buf], p, p2);
      } else if (unit != now_unit) {
#pragma unroll
        for (int i = 0; i < T::kParts; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][e] = __builtin_amdgcn_ldexpf(acc[i][e], unit - now_unit);
      }
      unit = now_unit;

      // values far below the step's largest: passes of their own, in place of the step's values
      if (now.v_least <= now_unit - kBand) {
        for (int band = 1; band < kBands && now_unit >= band * kBand; ++band) {
          const int ex = scale_exponent(now_unit - band * kBand);
          __syncthreads();
          if (for_values) {
#pragma unroll
            for (int u = 0; u < T::kUnits; ++u) {
              Staged again;
              load_codes(step, now_page[u], my_key + u * T::kUnitKeys, again);
              expand_values(step, now_page[u], my_key + u * T::kUnitKeys, again, lv[buf], ex, now_unit - band * kBand);
            }
          }
          __syncthreads();
          if (seen) {
#pragma unroll
            for (int i = 0; i < T::kParts; ++i)
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[i][e] = __builtin_amdgcn_ldexpf(acc[i][e], unit - ex);
            product(lv[buf], p, p2);
#pragma unroll
            for (int i = 0; i < T::kParts; ++i)
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[i][e] = __builtin_amdgcn_ldexpf(acc[i][e], ex - unit);
          }
        }
      }
      if (now.bad && seen) {
        for (int k = key0; k < key0 + T::kKeys && k < range.hi; ++k) {
          const int at_page = row_page(c.kv, table, c.rows.table_width, k);
          if (at_page < 0 || k > q_hi || k < q_lo) continue;
          const int64_t at = ((int64_t)at_page * H + h) * T::kGroups * ps + (k & (ps - 1));
#pragma unroll
          for (int gr = 0; gr < T::kGroups; ++gr) {
            if ((c.kv.p.k_scales[at + gr * ps] & 0x7F80) == 0x7F80) sum = NAN;
            if ((c.kv.p.v_scales[at + gr * ps] & 0x7F80) == 0x7F80)
#pragma unroll
              for (int i = 0; i < T::kParts; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if ((4 * i + e / 4) % T::kGroups == gr) acc[i][e] = NAN;
          }
        }
      }

      if (more) {
        const StepScales next = step_scales();
        const int e = scale_exponent(next.v);
        const int next_unit = e > now_unit || e < now_unit - kBand / 2 ? e : now_unit;
        expand_units(step + 1, page, g, buf ^ 1, scale_exponent(next.k), next_unit);
        now = next;
        now_unit = next_unit;
        there = __ballot(scale_page >= 0);
#pragma unroll
        for (int u = 0; u < T::kUnits; ++u) {
          now_page[u] = page[u];
          page[u] = page2[u];
        }
        scale_page = scale_page2;
      }
      __syncthreads();
    }

    sum += __shfl_xor(sum, 32);
    const float down = scale_unit(unit);
    const int64_t id = (int64_t)token * c.a.q_heads + head;
    const bool parts = c.prompt_splits > 1;
    // the share of the sum, or against the maximum, without the 2^7
    const float share = parts ? down * 0x1p-7f : sum != 0.0f ? down / sum : 0.0f;
    if (live) {
      uint16_t *out = static_cast<uint16_t *>(c.a.out) + token * c.a.out_token + head * c.a.out_head;
      float *part = c.part_o + (id * c.part_splits + split) * D;
      // columns 8 o .. 8 o + 7 are the rows b * kOct + o of V', b = 0 .. 7
#pragma unroll
      for (int k = 0; k < T::kParts * 2; ++k) {
        // k counts the o of this lane: bits of o below the lane half's, then those above
        const int o = 8 * (k / 4) + k % 4;  // + 4 hf
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = e * T::kOct + o, i = r / 32, rho = r % 32;
          v[e] = acc[i][rho / 8 * 4 + rho % 4] * share;
        }
        if (parts)
          __builtin_memcpy(part + 8 * (o + 4 * hf), v, 32);
        else
          store8(out, c.a.type, 8 * (o + 4 * hf), v);
      }
      if (hf == 0 && parts) c.part_ml[id * c.part_splits + split] = make_float2(m, sum * 0x1p-7f);
      if (hf == 0 && !parts && c.ml) c.ml[id] = make_float2(m, sum * 0x1p-7f);
    }
  }
}

template <int D>
hipError_t launch_d(const Call &c, hipStream_t s) {
  const int64_t tiles = (int64_t)c.rows.tokens * c.group / Prompt<D>::kRows + c.rows.seqs;
  const int64_t work = tiles * c.kv.p.kv_heads * c.prompt_splits;
  const auto kernel = c.a.type == COLI_MOE_F16 ? kv_prompt_kernel<D, true> : kv_prompt_kernel<D, false>;
  return launch(kernel, dim3((unsigned)(work < (1 << 20) ? work : 1 << 20)), dim3(Prompt<D>::kThreads), 0, s, c, work);
}

}  // namespace

hipError_t launch_attention_prompts(const Call &c, hipStream_t s) {
  switch (c.kv.p.head_dim) {
    case 64: return launch_d<64>(c, s);
    case 128: return launch_d<128>(c, s);
    default: return launch_d<256>(c, s);
  }
}

}  // namespace coli
