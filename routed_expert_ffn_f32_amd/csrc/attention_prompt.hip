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
// the values of each step.  A key whose scale is more than 25 powers of two
// below another's of its step has its scores computed apart.  Where the scales of
// a step's values are more than 25 powers of two apart, the small ones follow in
// passes of their own, so a value counts down to 2^-77 of the largest next to it,
// or 2^-100 of the largest before it.  Rows whose scale is NaN (or Inf) stay out
// of the products, where 0 times NaN would reach rows that do not see them, and
// are put on those that do.
//
// Bound by the sum of two units' work, of which too little runs at once: the
// vector units are busy for 51 % of the time and the matrix cores for 33 (a
// wave's step of 64 keys has 64 matrix instructions of 32 cycles and about 350
// vector ones of 4, of which 32 exponentials take 16, beside 190 scalar; one
// barrier a step keeps the waves of a SIMD in the same phase).  Two prompts of up
// to 1500 tokens on up to 16384 rows, 64 query heads on 8 of 128 columns: 1.55 ms,
// 625 TFLOP/s (a large product of the library's: 1.17 PFLOP/s); with all work in
// its order, before the scores of the next 32 keys went beside the weights of
// these, 1.85; by the tiles of a few rows 5.5.  D = 64 runs at 370, D = 256, whose
// results and queries leave one workgroup of four waves a CU its registers, at
// 280.
#include "attention.h"

namespace coli {
namespace {

typedef float float16_t __attribute__((ext_vector_type(16)));

constexpr int kBand = 26;    // powers of two of one pass over the values
constexpr int kBands = 3;
template <int N>
struct Num {
  static constexpr int value = N;
};

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
  // Half of the waves expand values, the others keys.  A lane's unit is 8
  // columns of 4 keys' values, or 32 columns (D = 64: 16) of one key; a wave's
  // lanes stay within 16 keys, which share a page.
  static constexpr int kStageWaves = kWaves / 2;
  static constexpr int kPieces = D == 64 ? 4 : D / 32;       // of a key's row
  static constexpr int kWaveKeys = D == 256 ? 8 : 16;        // of a wave's unit
  static constexpr int kUnitKeys = kStageWaves * kWaveKeys;  // from one unit to the next
  static constexpr int kUnits = kKeys / kUnitKeys;           // of a lane
  static_assert(kUnits >= 1 && kUnitKeys * kUnits == kKeys && kWaveKeys * kPieces == 64, "units cover a step");
};

__device__ __forceinline__ int wave_max(int v) {
  v = max(v, dpp_i<kDppQuadXor1>(v));
  v = max(v, dpp_i<kDppQuadXor2>(v));
  v = max(v, dpp_i<kDppRowRor4>(v));
  v = max(v, dpp_i<kDppRowRor8>(v));
  return max(max(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
             max(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}

// The larger of a lane's and of the lane's 32 away.
__device__ __forceinline__ float max_over_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Exponents of the scales of a step: largest of the keys' and the smallest that
// is a key's largest, largest and smallest of the values' (none of 0), and
// whether one is NaN or Inf.
struct StepScales {
  int k, v, v_least, k_least;
  bool bad;
  uint64_t there;  // keys that are on a page
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

// A unit of a step as it stands in memory, and values' codes with their scales.
struct Staged {
  u32x4 code;
  uint2 scale;
};
struct ValueUnit {
  uint32_t code[4];
  half2_t scale[2];
};

template <int D, bool kTwice>
__global__ __launch_bounds__(Prompt<D>::kThreads, D == 256 ? 1 : 2) void kv_prompt_kernel(Call c, int64_t work) {
  using T = Prompt<D>;
  // keys of the step, of the next (whose first scores are computed beside this one's last) and of the one after
  __shared__ __align__(16) _Float16 lk[3][T::kKeys * T::kKeyRow];
  __shared__ __align__(16) _Float16 lv[2][D * T::kValRow];
  __shared__ uint4 told[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), hf = lane >> 5, l32 = lane & 31;
  const int H = c.kv.p.kv_heads, ps = c.kv.p.page_size, S = c.rows.seqs;

  // a call that may have prompts but has none is over here (8 sequences of 8 tokens: 13.6 us without)
  if (S <= 64) {
    const SeqSpan mine = seq_span(c.rows, min(lane, S - 1));
    if (!__any(mine.n * c.group > c.few_rows)) return;
  }
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
    // keys are numbers up to 2^30
    const int first_key = (int)min(range.lo, (int64_t)1 << 30) & ~(T::kKeys - 1), end_key = (int)max(range.hi, (int64_t)0);
    const int steps = range.hi > range.lo ? (end_key - first_key + T::kKeys - 1) / T::kKeys : 0;
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
    auto clamped = [](int64_t v) { return (int)min(max(v, (int64_t)-1), (int64_t)1 << 30); };
    const int64_t pos0 = len - span.n + w0 / c.group, pos1 = len - span.n + w1 / c.group;
    const int p0 = clamped(pos0);
    const int all_lo = c.a.window ? clamped(pos1 - c.a.window + 1) : 0;

    half8_t q[T::kSteps];
    float q_unit;
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
      q_unit = unlift(ex);
    }

    float16_t acc[T::kParts];
#pragma unroll
    for (int i = 0; i < T::kParts; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
    float m = -INFINITY, sum = 0.0f;  // the maximum that the sums stand against; the sum of 2^7 times the weights
    bool far = false;                 // a row's maximum is above kFar

    // --- staging ---
    const bool for_values = wave < T::kStageWaves;
    // values: keys 4 quad .. + 3 (of the wave's), columns 8 oct .. + 7 (D = 64 has fewer units than lanes);
    // keys: columns 32 (D = 64: 16) piece .. of one key
    const int oct = lane % T::kOct, quad = lane / T::kOct, piece = lane % T::kPieces;
    const bool stages = !for_values || 4 * quad < T::kWaveKeys;
    const int wave_key = wave % T::kStageWaves * T::kWaveKeys;        // of the step, for the first unit
    const int lane_key = for_values ? 4 * quad % T::kWaveKeys : lane / T::kPieces;  // from there on

    // Page of key k of a step: the table's entry as it stands, so that the load
    // need not be waited for, and later -1 where there is none or none is seen.
    const int last_page = c.rows.table_width - 1;
    auto page_entry = [&](int step, int k) {
      return table[min((first_key + step * T::kKeys + k) >> c.kv.shift, last_page)];
    };
    auto page_checked = [&](int step, int k, int entry) {
      return step < s1 && first_key + step * T::kKeys + k < end_key && (unsigned)entry < (unsigned)c.kv.p.n_pages ? entry
                                                                                                               : -1;
    };
    // The scales of a step: one wave looks at them, a key a lane, two steps ahead,
    // and tells the others through LDS.
    const int scale_key = lane % T::kKeys;
    struct Scales {
      uint16_t k[T::kGroups], v[T::kGroups];
    };
    auto load_scales = [&](int step, int page, Scales &to) {
      const int slot = (first_key + step * T::kKeys + scale_key) & (ps - 1);
#pragma unroll
      for (int g = 0; g < T::kGroups; ++g) {
        const uint64_t at = scale_index<T::kGroups>(c.kv, max(page, 0), h, g, slot);
        to.k[g] = c.kv.p.k_scales[at];
        to.v[g] = c.kv.p.v_scales[at];
      }
    };
    auto tell_scales = [&](int step, int page, const Scales &from) {
      int k = 0, v = 0, least = 254;
      bool bad = false, some = false;
#pragma unroll
      for (int g = 0; g < T::kGroups; ++g) {
        const int bk = page < 0 ? 0 : from.k[g], bv = page < 0 ? 0 : from.v[g];
        const int ek = bk >> 7 & 255, ev = bv >> 7 & 255;
        bad = bad || ek == 255 || ev == 255;
        k = max(k, ek == 255 ? 0 : ek);
        some = some || (bk & 0x7FFF) != 0;
        v = max(v, ev == 255 ? 0 : ev);
        least = min(least, (bv & 0x7FFF) == 0 || ev == 255 ? 254 : ev);
      }
      const uint64_t there = __ballot(page >= 0);
      const int any_bad = __any(bad) ? 1 << 24 : 0;
      const int k_least = 254 - wave_max(254 - (some ? k : 254));
      k = wave_max(k);
      v = wave_max(v);
      least = 254 - wave_max(254 - least);
      if (lane == 0)
        told[(step - s0) & 3] = make_uint4(k | v << 8 | least << 16 | any_bad, k_least, (uint32_t)there,
                                           (uint32_t)(there >> 32));
    };
    auto hear_scales = [&](int step) {
      const uint4 t = told[(step - s0) & 3];
      const int packed = uniform((int)t.x);
      StepScales r;
      r.k = packed & 255;
      r.v = packed >> 8 & 255;
      r.v_least = packed >> 16 & 255;
      r.bad = packed >> 24;
      r.k_least = uniform((int)t.y);
      r.there = (uint32_t)uniform((int)t.z) | (uint64_t)(uint32_t)uniform((int)t.w) << 32;
      return r;
    };
    // Codes and scales of a unit, by the same loads for keys and values: from a
    // uniform address, a lane's own few bytes on.
    const int lane_byte = lane_key * (D / 2) + (for_values ? 4 * oct : (D == 64 ? 8 : 16) * piece);
    const int lane_scale = (for_values ? oct / 8 : piece * (D == 64 ? 16 : 32) / kKvGroup) * ps + (lane_key & ~3);
    const uint8_t *codes = for_values ? c.kv.p.v_codes : c.kv.p.k_codes;
    const uint16_t *scales = for_values ? c.kv.p.v_scales : c.kv.p.k_scales;
    auto load_codes = [&](int step, int page, int unit_key, Staged &g) {
      const int slot = (first_key + step * T::kKeys + unit_key) & (ps - 1);
      const uint8_t *base = codes + code_row(c.kv, max(page, 0), h, slot) * (D / 2);
#pragma unroll
      for (int i = 0; i < 4; ++i)  // D = 64: a key has two dwords
        g.code[i] = *reinterpret_cast<const uint32_t *>(
            base + (lane_byte + (for_values ? i * (D / 2) : (D == 64 ? i & 1 : i) * 4)));
      // four keys from a multiple of four on
      g.scale = *reinterpret_cast<const uint2 *>(scales + scale_index<T::kGroups>(c.kv, max(page, 0), h, 0, slot & ~3) +
                                                 lane_scale);
    };
    // Scales of a unit as halves: of its keys that are before the range's end and on
    // a page, else 0.  Then its codes times them, in 8 pieces (values: a row of V'
    // each; keys: 4, the even ones, a dword each).
    auto value_unit = [&](int step, int page, int unit_key, const Staged &g, int ex, int limit) {
      const int k0 = first_key + step * T::kKeys + unit_key + lane_key;
      const float up = scale_up(ex);
      ValueUnit r;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t two = i ? g.scale.y : g.scale.x;
        const uint32_t a = page >= 0 && k0 + 2 * i < end_key ? two & 0xFFFFu : 0u;
        const uint32_t d = page >= 0 && k0 + 2 * i + 1 < end_key ? two >> 16 : 0u;
        r.scale[i] = half2_t{val_scale(a, up, limit), val_scale(d, up, limit)};
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) r.code[i] = g.code[i];
      return r;
    };
    auto expand_values = [&](const ValueUnit &r, int unit_key, _Float16 *to, int i) {
      if (!stages) return;
      const uint32_t sel = 0x0C040C00u + 0x00010001u * (i / 2);
      const uint32_t t0 = __builtin_amdgcn_perm(r.code[1], r.code[0], sel);
      const uint32_t t1 = __builtin_amdgcn_perm(r.code[3], r.code[2], sel);
      // keys 0-3, 4-7, 8-11, 12-15 of 16 stand in the order 0-3, 8-11, 4-7, 12-15
      const int at = (unit_key + lane_key) / 4, chunk = at / 4 * 2 + (at & 1), half = at >> 1 & 1;
      *reinterpret_cast<uint2 *>(to + (i * T::kOct + oct) * T::kValRow + 8 * chunk + 4 * half) =
          i & 1 ? make_uint2(times(high_codes(t0), r.scale[0]), times(high_codes(t1), r.scale[1]))
                : make_uint2(times(low_codes(t0), r.scale[0]), times(low_codes(t1), r.scale[1]));
    };
    auto key_unit = [&](int step, int page, int unit_key, const Staged &g, int ex) {
      const int k0 = first_key + step * T::kKeys + unit_key + lane_key;
      const uint32_t two = k0 & 2 ? g.scale.y : g.scale.x, mine = k0 & 1 ? two >> 16 : two & 0xFFFFu;
      const _Float16 one = key_scale(page >= 0 && k0 < end_key ? mine : 0u, scale_up(ex));
      return half2_t{one, one};
    };
    auto expand_keys = [&](half2_t s, int unit_key, const Staged &g, _Float16 *to, int i) {
      if (D == 64 && i > 1) return;
      u32x4 v = __builtin_bit_cast(u32x4, codes_of(g.code[i]));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = times(v[e], s);
      *reinterpret_cast<u32x4 *>(to + (unit_key + lane_key) * T::kKeyRow + 8 * (piece * (D == 64 ? 2 : 4) + i)) = v;
    };
    // The two products.  A matrix instruction is under way for 32 cycles after the
    // 4 of its issue, so vector work is put between them: work(n) follows
    // instruction n, and the scheduler is kept from moving what stands between two
    // of them (left alone it gathers the vector work behind the last).  Operands
    // are read kLead instructions ahead.
    constexpr int kLead = 4;
    auto product = [&](const _Float16 *from, int sub, const half8_t (&p)[2], const half8_t (&p2)[2], auto work) {
      constexpr int kCount = 2 * T::kParts;
      half8_t a[kLead];
      auto read = [&](int n) {
        const int u = 2 * sub + n / T::kParts, i = n % T::kParts;
        return *reinterpret_cast<const half8_t *>(from + (32 * i + l32) * T::kValRow + 8 * (2 * u + hf));
      };
#pragma unroll
      for (int n = 0; n < kLead; ++n) a[n] = read(n);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < kCount; ++n) {
        const int u = n / T::kParts, i = n % T::kParts;
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[n % kLead], p[u], acc[i], 0, 0, 0);
        if constexpr (kTwice) acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[n % kLead], p2[u], acc[i], 0, 0, 0);
        if (n + kLead < kCount) a[n % kLead] = read(n + kLead);
        work(n);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto scores = [&](const _Float16 *from, int sub, float16_t &x, auto work) {
      half8_t a[kLead];
      auto read = [&](int n) {
        return *reinterpret_cast<const half8_t *>(from + (32 * sub + l32) * T::kKeyRow + 8 * (2 * n + hf));
      };
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.0f;
#pragma unroll
      for (int n = 0; n < kLead; ++n) a[n] = read(n);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < T::kSteps; ++n) {
        x = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[n % kLead], q[n], x, 0, 0, 0);
        if (n + kLead < T::kSteps) a[n % kLead] = read(n + kLead);
        work(n);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    // all units of this lane
    auto pages_of = [&](int step, int (&to)[T::kUnits]) {
#pragma unroll
      for (int u = 0; u < T::kUnits; ++u) to[u] = page_entry(step, wave_key + lane_key + u * T::kUnitKeys);
    };
    auto check_pages = [&](int step, int (&pages)[T::kUnits]) {
#pragma unroll
      for (int u = 0; u < T::kUnits; ++u)
        pages[u] = page_checked(step, wave_key + u * T::kUnitKeys, uniform(pages[u]));
    };
    auto load_units = [&](int step, const int (&pages)[T::kUnits], Staged (&to)[T::kUnits]) {
#pragma unroll
      for (int u = 0; u < T::kUnits; ++u) load_codes(step, pages[u], wave_key + u * T::kUnitKeys, to[u]);
    };
    auto expand_units = [&](int step, const int (&pages)[T::kUnits], const Staged (&from)[T::kUnits], _Float16 *values_to,
                            _Float16 *keys_to, int k_ex, int v_ex, int limit) {
#pragma unroll
      for (int u = 0; u < T::kUnits; ++u) {
        const int unit_key = wave_key + u * T::kUnitKeys;
        if (for_values) {
          const ValueUnit r = value_unit(step, pages[u], unit_key, from[u], v_ex, limit);
#pragma unroll
          for (int i = 0; i < 8; ++i) expand_values(r, unit_key, values_to, i);
        } else {
          const half2_t scale = key_unit(step, pages[u], unit_key, from[u], k_ex);
#pragma unroll
          for (int i = 0; i < 4; ++i) expand_keys(scale, unit_key, from[u], keys_to, i);
        }
      }
    };

    // Step t expands the values of t + 1 and the keys of t + 2.  Within it, 32 keys
    // at a time: the scores of the next 32 beside the weights of these, then their
    // product beside a share of the expansion.
    const int ahead = for_values ? 1 : 2;
    int unit = 12;      // exponent of the values' power of two that acc stands in
    int now_unit = 12;  // and that the step's values are expanded to
    int next_unit = 12;
    int top_unit = 12;  // the largest so far
    int k_now = 0, k_next = 1, k_after = 2;  // whose keys stand where
    StepScales now = {12, 12, 254, 254, false, 0}, next = now, next2 = now;
    Staged g[T::kUnits];
    int page[T::kUnits], page2[T::kUnits], now_page[T::kUnits], look_page = -1;
    float16_t xa, xb;
    __syncthreads();  // of the item before, all is read
    if (s0 < s1) {
      pages_of(s0, page);
      check_pages(s0, page);
      load_units(s0, page, g);
      if (wave < 3) {
        const int at = page_checked(s0 + wave, scale_key, page_entry(s0 + wave, scale_key));
        Scales sc;
        load_scales(s0 + wave, at, sc);
        tell_scales(s0 + wave, at, sc);
      }
      __syncthreads();
      now = hear_scales(s0);
      next = hear_scales(s0 + 1);
      unit = now_unit = top_unit = scale_exponent(now.v);
      expand_units(s0, page, g, lv[0], lk[0], scale_exponent(now.k), now_unit, now_unit);
#pragma unroll
      for (int u = 0; u < T::kUnits; ++u) now_page[u] = page[u];
      if (!for_values) {
        pages_of(s0 + 1, page);
        check_pages(s0 + 1, page);
        load_units(s0 + 1, page, g);
        expand_units(s0 + 1, page, g, lv[1], lk[1], scale_exponent(next.k), 12, 12);
      }
      pages_of(s0 + ahead, page);
      if ((s0 & (T::kWaves - 1)) == wave) look_page = page_entry(s0 + 3, scale_key);
      __syncthreads();
      scores(lk[0], 0, xa, [](int) {});
    }
    Scales look;
    ValueUnit expanding;

    auto begin_step = [&](int step) {
      check_pages(step + ahead, page);
      load_units(step + ahead, page, g);
      pages_of(step + ahead + 1, page2);
      // one wave in turn looks at the scales of step + 3, with the pages that it
      // has asked for a step before
      if ((step & (T::kWaves - 1)) == wave) {
        look_page = page_checked(step + 3, scale_key, look_page);
        load_scales(step + 3, look_page, look);
      }
      next2 = hear_scales(step + 2);
      // A step of much smaller values has a smaller unit, but not one that sums of
      // the largest so far would overflow in; one without values has none of its own.
      const int e1 = next.v == 0 ? now_unit : scale_exponent(next.v);
      next_unit = e1 > now_unit || e1 < now_unit - kBand / 2 ? max(e1, top_unit - kBand) : now_unit;
      top_unit = max(top_unit, next_unit);
    };
    auto end_step = [&](int step) {
      if ((step & (T::kWaves - 1)) == wave) tell_scales(step + 3, look_page, look);
      if ((step + 1 & (T::kWaves - 1)) == wave) look_page = page_entry(step + 4, scale_key);
      now = next;
      next = next2;
      now_unit = next_unit;
      const int free_keys = k_now;
      k_now = k_next;
      k_next = k_after;
      k_after = free_keys;
#pragma unroll
      for (int u = 0; u < T::kUnits; ++u) {
        now_page[u] = page[u];
        page[u] = page2[u];
      }
      __syncthreads();
    };
    // keys 32 sub .. of a step, whose scores are x; y: those of the next 32
    auto half_step = [&](int step, auto sub_of, float16_t &x, float16_t &y) {
      constexpr int sub = decltype(sub_of)::value;
      const int buf = (step - s0) & 1;
      const int key0 = first_key + step * T::kKeys + 32 * sub;
      const uint32_t there = (uint32_t)(now.there >> (32 * sub));
      const int k_ex = scale_exponent(now.k);
      // keys far below the step's largest, which a row may not even see: their scores from the codes as they stand
      if (__builtin_expect(now.k_least <= k_ex - kBand, 0)) {
        for (int k = 0; k < 32; ++k) {
          const int page = key0 + k < end_key ? row_page(c.kv, table, c.rows.table_width, key0 + k) : -1;
          if (page < 0) continue;
          const int slot = (key0 + k) & (ps - 1);
          const uint32_t *code =
              reinterpret_cast<const uint32_t *>(c.kv.p.k_codes + code_row(c.kv, page, h, slot) * (D / 2));
          const uint16_t *sc = c.kv.p.k_scales + scale_index<T::kGroups>(c.kv, page, h, 0, slot);
          int own = 0;
#pragma unroll
          for (int gr = 0; gr < T::kGroups; ++gr) own = max(own, sc[gr * ps] >> 7 & 255);
          if (own > k_ex - kBand) continue;  // in the product, or NaN
          float total = 0.0f;
#pragma unroll
          for (int n = 0; n < T::kSteps; ++n) {
            __builtin_amdgcn_sched_barrier(0);  // one after the other: registers are short
            const half8_t v = codes_of(code[2 * n + hf]);
            float part = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) part = __builtin_fmaf((float)v[e], (float)q[n][e], part);
            total = __builtin_fmaf(part, from_bf16(sc[16 * n / kKvGroup * ps]) * scale_up(k_ex), total);
          }
          total += __shfl_xor(total, 32);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = k == 8 * (e / 4) + e % 4 + 4 * hf ? total : x[e];
        }
      }
      if (__builtin_expect(!(key0 + 31 <= p0 && key0 >= all_lo && there == ~0u), 0)) {
        const uint32_t mine = there >> (4 * hf);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int at = 8 * (e / 4) + e % 4, k = key0 + at + 4 * hf;
          x[e] = k <= q_hi && k >= q_lo && (mine >> at & 1) ? x[e] : -INFINITY;
        }
      }
      // more than 0, so that masked scores stay what they are
      const float f = fmaxf(q_unit * scale_unit(k_ex), 0x1p-126f);
      float top = x[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, x[e]);
      top = max_over_halves(top) * f;
      if (__builtin_expect(__any((top - m) * c.cs > kSlack) || unit != now_unit, 0)) {
        const float m1 = fmaxf(m, top);
        const float fade = __builtin_amdgcn_exp2f((m - (m1 == -INFINITY ? 0.0f : m1)) * c.cs);
        m = m1;
        far = __any(fabsf(m) * c.cs > kFar && m != -INFINITY);
        sum *= fade;
#pragma unroll
        for (int i = 0; i < T::kParts; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][e] = __builtin_amdgcn_ldexpf(acc[i][e] * fade, unit - now_unit);
        unit = now_unit;
      }
      const float base = m == -INFINITY ? 0.0f : m;
      float by = fmaxf(f * c.cs, 0x1p-126f), plus = __builtin_fmaf(-base, c.cs, 7.0f);
      if (__builtin_expect(far, 0)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __builtin_fmaf(x[e], f, -base);
        by = c.cs;
        plus = 7.0f;
      }
      half8_t p[2], p2[2];
      // weights: kEach exponentials after an instruction, and the sum and rounding of those before
      constexpr int kEach = (16 + T::kSteps - 1) / T::kSteps;
      float v[2][kEach];
      auto settle = [&](int n) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const int at = n * kEach + j;
          sum += v[n & 1][j];
          const _Float16 hi = (_Float16)v[n & 1][j];
          p[at / 8][at % 8] = hi;
          if constexpr (kTwice) p2[at / 8][at % 8] = (_Float16)(v[n & 1][j] - (float)hi);
        }
      };
      const bool last = sub + 1 == T::kSubs;
      scores(lk[last ? k_next : k_now], last ? 0 : sub + 1, y, [&](int n) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const int at = n * kEach + j;
          v[n & 1][j] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[at], by, plus));
        }
        if (n > 0) settle(n - 1);
      });
      settle(T::kSteps - 1);
      // the expansion in this half's share of the 8 pieces of each unit
      constexpr int kWork = 8 * T::kUnits / T::kSubs, kProduct = 2 * T::kParts;
      auto pieces = [&](int n, auto expand) {
        // piece j after instruction j kProduct / kWork
#pragma unroll
        for (int j = 0; j < kWork; ++j)
          if (j * kProduct / kWork == n) expand(sub * kWork + j);
      };
      product(lv[buf], sub, p, p2, [&](int n) {
        pieces(n, [&](int k) {
          const int u = k / 8, unit_key = wave_key + u * T::kUnitKeys;
          if (for_values) {
            if (k % 8 == 0) expanding = value_unit(step + 1, page[u], unit_key, g[u], next_unit, next_unit);
            expand_values(expanding, unit_key, lv[buf ^ 1], k % 8);
          } else {
            if (k % 8 == 0) expanding.scale[0] = key_unit(step + 2, page[u], unit_key, g[u], scale_exponent(next2.k));
            if (k % 2 == 0) expand_keys(expanding.scale[0], unit_key, g[u], lk[k_after], k % 8 / 2);
          }
        });
      });
      // values far below the step's largest: passes of their own, in place of the step's values, which the last one
      // puts back for the step's other half
      if (__builtin_expect(now.v_least <= now_unit - kBand, 0)) {
        const int bands = min(kBands, now_unit / kBand + 1);
        for (int band = 1; band <= bands; ++band) {
          const int limit = band < bands ? now_unit - band * kBand : now_unit, ex = scale_exponent(limit);
          __syncthreads();
          if (for_values) {
            Staged again[T::kUnits];
            load_units(step, now_page, again);
            expand_units(step, now_page, again, lv[buf], lk[0], 12, ex, limit);
          }
          __syncthreads();
          if (band == bands) break;
#pragma unroll
          for (int i = 0; i < T::kParts; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][e] = __builtin_amdgcn_ldexpf(acc[i][e], unit - ex);
          product(lv[buf], sub, p, p2, [](int) {});
#pragma unroll
          for (int i = 0; i < T::kParts; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][e] = __builtin_amdgcn_ldexpf(acc[i][e], ex - unit);
        }
      }
      if (__builtin_expect(now.bad, 0)) {
        for (int k = key0; k < key0 + 32 && k < end_key; ++k) {
          const int at_page = row_page(c.kv, table, c.rows.table_width, k);
          if (at_page < 0 || k > q_hi || k < q_lo) continue;
#pragma unroll
          for (int gr = 0; gr < T::kGroups; ++gr) {
            const uint64_t at = scale_index<T::kGroups>(c.kv, at_page, h, gr, k & (ps - 1));
            if ((c.kv.p.k_scales[at] & 0x7F80) == 0x7F80) sum = NAN;
            if ((c.kv.p.v_scales[at] & 0x7F80) == 0x7F80)
#pragma unroll
              for (int i = 0; i < T::kParts; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if ((4 * i + e / 4) % T::kGroups == gr) acc[i][e] = NAN;
          }
        }
      }
    };
    for (int step = s0; step < s1; ++step) {
      begin_step(step);
      half_step(step, Num<0>{}, xa, xb);
      if constexpr (T::kSubs == 2) {
        half_step(step, Num<1>{}, xb, xa);
        end_step(step);
      } else {
        end_step(step);
        if (++step >= s1) break;
        begin_step(step);
        half_step(step, Num<0>{}, xb, xa);
        end_step(step);
      }
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
