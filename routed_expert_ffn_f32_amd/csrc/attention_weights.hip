// The attention weights of cached rows where sequences have more rows of
// queries than one tile of the attention's: for every key the sum over the
// query rows of its key head of
//   exp2((q . k - m) cs) / l
// with the rows' maxima m and sums l that the attention has left.
//
// A product whose result is summed over the queries at once: each wave holds 64
// keys (D = 256: 32) as the left operand for good, the query rows come by in
// tiles of 32 through LDS, and the sums of a key stay in its registers, one for
// each query column, until the end.  A key has a power of two of its own, so
// its codes times its scales are exact.  Bound by what follows the product (an
// exponential and four operations an element, 32 cycles to the product's 16 at
// D = 128), so queries are made halves once by a kernel of their own, and the
// tiles that all rows see whole have no masks.  Two prompts of up to 1500 tokens
// on up to 16384 rows, 64 query heads on 8 of 128 columns: 1.2 ms; by the tiles
// of the attention, a tile's scores once more for each 64 keys, 6.2.
#include "attention.h"
#include "lds_dma.h"

namespace coli {
namespace {

typedef float float16_t __attribute__((ext_vector_type(16)));

constexpr int kRowTile = 32;
constexpr int kWaves = 8;
constexpr int kRing = 3;

// Queries as halves after a power of two per row, 8 columns in the order of
// codes_of, the 16-byte pieces of a row exchanged by its index so that rows
// side by side in LDS are read without conflicts.
template <int D>
__global__ __launch_bounds__(256) void kv_weight_rows_kernel(Call c, int64_t rows) {
  constexpr int kPieces = D / 8;
  const int64_t total = rows * kPieces, step = (int64_t)gridDim.x * 256;
  // whole waves: rows are not divided between them
  for (int64_t x0 = (int64_t)blockIdx.x * 256 + (threadIdx.x & ~63); x0 < total; x0 += step) {
    const int64_t x = x0 + (threadIdx.x & 63), id = min(x / kPieces, rows - 1);
    const int piece = threadIdx.x % kPieces, head = (int)(id % c.a.q_heads);
    const int64_t token = id / c.a.q_heads;
    const char *from = static_cast<const char *>(c.a.q) + (token * c.a.q_token + head * c.a.q_head + piece * 8) * 2;
    const u32x4 raw = load16(from);
    float v[8], top = 0.0f;
    unpack8(c.a.type, Raw8{raw, raw}, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
    for (int d = 1; d < kPieces; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    const int ex = lift_exponent(top);
    const float up = c.a.scale > 0.0f ? lift(ex) : c.a.scale < 0.0f ? -lift(ex) : 0.0f;
    half8_t y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[2 * e] = (_Float16)(v[e] * up);
      y[2 * e + 1] = (_Float16)(v[e + 4] * up);
    }
    if (x >= total) continue;
    const int64_t in_head = token * c.group + head % c.group;
    const int64_t row = (int64_t)(head / c.group) * c.rows.tokens * c.group + in_head;
    *reinterpret_cast<half8_t *>(c.q_halves + row * (2 * D) + (piece ^ (int)(in_head & 7)) * 16) = y;
    if (piece == 0) {
      const float2 ml = c.ml[id];
      c.q_info[row] = make_float4(unlift(ex), ml.x == -INFINITY ? 0.0f : ml.x, share_again(ml.y),
                                  limit_again(ml.y));
    }
  }
}

// kTiles: of 32 keys a wave.
template <int D, int kTiles, bool kSmallPages>
__global__ __launch_bounds__(64 * kWaves, 2) void kv_row_weights_kernel(Call c, int64_t work) {
  constexpr int kKeys = kWaves * 32 * kTiles;
  constexpr int kSteps = D / 16, kGroups = D / kKvGroup;
  constexpr int kTileBytes = kRowTile * D * 2, kInfoBytes = kRowTile * 16;
  constexpr int kCopies = kTileBytes / 1024;  // of a tile of queries, by all waves
  __shared__ __align__(16) char ring[kRing][kTileBytes + kInfoBytes];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 31, hf = lane >> 5;
  const int H = c.kv.p.kv_heads;
  const int64_t sh = (int64_t)c.rows.seqs * H;
  // a wave's copies of a tile: the last one's also the rows' numbers
  const int mine = (wave < kCopies ? (kCopies + kWaves - 1) / kWaves : 0) + (wave == kWaves - 1 ? 1 : 0);
  // sequences and heads first: the workgroups that read the same queries are on one XCD
  for (int64_t item = blockIdx.x; item < work; item += gridDim.x) {
    const int h = (int)(item % H), s = (int)(item % sh / H);
    const SeqSpan span = seq_span(c.rows, s);
    const int64_t len = c.rows.lengths[s], start = len - span.n;
    const int64_t end = min(len, (int64_t)c.rows.table_width << c.kv.shift);
    const int rows = span.n * c.group;
    if (rows == 0) continue;
    // a table may be far wider than its sequence: the parts go on to the sequence's end
    for (int64_t key_at = item / sh * kKeys; key_at < end; key_at += work / sh * kKeys) {
      const int key0 = (int)key_at;
      // queries that see any of these keys
      const int64_t i0 = max((int64_t)key0 - start, (int64_t)0);
      const int64_t i1 = c.a.window ? min(key0 + kKeys - 1 + (int64_t)c.a.window - start, (int64_t)span.n)
                                    : (int64_t)span.n;
      if (i0 >= i1) continue;
      const int first = (int)(i0 * c.group / kRowTile), last = (int)((i1 * c.group - 1) / kRowTile);
      const int64_t row0 = (int64_t)h * c.rows.tokens * c.group + (int64_t)span.first * c.group;
      const int swap = (span.first * c.group + r) & 7;
      auto copy = [&](int tile, int slot) {
        const uint32_t to = uniform(lds_addr(ring[slot]));
        const char *q = c.q_halves + (row0 + (int64_t)tile * kRowTile) * (2 * D);
#pragma unroll
        for (int i = 0; i < (kCopies + kWaves - 1) / kWaves; ++i) {
          const int part = i * kWaves + wave;
          if (part < kCopies) dma16v(to + part * 1024, q + part * 1024 + lane * 16);
        }
        if (wave == kWaves - 1 && lane < 32)
          dma16v(to + kTileBytes, reinterpret_cast<const char *>(c.q_info + row0 + (int64_t)tile * kRowTile) + lane * 16);
      };

      const int32_t *table = c.rows.table + s * c.rows.table_stride;
      const int keys0 = key0 + wave * 32 * kTiles;
      const int off = kSmallPages ? r & 15 : r, half = r >> 4;  // where this lane's key is
      half8_t a[kTiles][kSteps];
      float fk[kTiles][16];
      uint64_t at[kTiles];
      bool ok[kTiles];
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        const int key = keys0 + 32 * u;
        const Place<kSmallPages> p = place_of<D, kSmallPages>(c, entries_of<kSmallPages>(c, table, key), h, key);
        at[u] = p.row[kSmallPages ? half : 0] + off;
        ok[u] = half ? p.ok[1] : p.ok[0];
        u32x4 codes[D / 64];
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          codes[i] = load16(reinterpret_cast<const char *>(c.kv.p.k_codes) + at[u] * (D / 2) + hf * (D / 4) + 16 * i);
        // this half's scales: D = 64 one for both, 128 one each, 256 two each
        constexpr int kOwn = D == 256 ? 2 : 1;
        float sc[kOwn], top = 0.0f;
        bool bad = false;
#pragma unroll
        for (int g = 0; g < kOwn; ++g) {
          const int group = kGroups == 1 ? 0 : hf * kOwn + g;
          sc[g] = from_bf16(c.kv.p.k_scales[p.scale[kSmallPages ? half : 0] + ((uint64_t)group << c.kv.shift) + off]);
          const bool finite = (__float_as_uint(sc[g]) & 0x7F800000u) != 0x7F800000u;
          bad = bad || !finite;
          sc[g] = finite ? sc[g] : 0.0f;
          top = fmaxf(top, fabsf(sc[g]));
        }
        top = fmaxf(top, __shfl_xor(top, 32));
        bad = bad || __shfl_xor((int)bad, 32);
        // codes times scale are 11 bits, exact as halves below 2^15
        const int ex = lift_exponent(top);
#pragma unroll
        for (int n = 0; n < kSteps; ++n) {
          const _Float16 by = (_Float16)(sc[D == 256 ? n / 8 : 0] * lift(ex) * 0x1p-4f);
          a[u][n] = codes_of(codes[n / 4][n % 4]) * half8_t{by, by, by, by, by, by, by, by};
        }
        const float back = bad ? NAN : unlift(ex) * 0x1p4f;
#pragma unroll
        for (int i = 0; i < 16; ++i) fk[u][i] = __shfl(back, 8 * (i / 4) + 4 * hf + i % 4);
      }

      float sum[kTiles][16] = {};
      __syncthreads();  // of the item before, all is read
      copy(first, 0);
      if (first < last) copy(first + 1, 1);
      int slot = 0;
      for (int tile = first; tile <= last; ++tile) {
        if (tile == last)
          dma_wait<0>();
        else if (mine == 1)
          dma_wait<1>();
        else if (mine == 2)
          dma_wait<2>();
        else
          dma_wait<3>();
        __syncthreads();
        if (tile + 2 <= last) copy(tile + 2, slot == 0 ? 2 : slot - 1);
        const char *q = ring[slot];
        slot = slot == kRing - 1 ? 0 : slot + 1;
        // positions of the tile's rows: from p0 up to p1 at most
        const int i_first = tile * kRowTile / c.group;
        const int64_t p0 = start + i_first, p1 = min(p0 + (kRowTile - 1) / c.group + 1, len - 1);
        if (keys0 > p1) continue;
        float16_t x[kTiles] = {};
#pragma unroll
        for (int n = 0; n < kSteps; ++n) {
          const half8_t b = *reinterpret_cast<const half8_t *>(q + r * (2 * D) + ((hf * kSteps + n) ^ swap) * 16);
#pragma unroll
          for (int u = 0; u < kTiles; ++u) x[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[u][n], b, x[u], 0, 0, 0);
        }
        const float4 f = *reinterpret_cast<const float4 *>(q + kTileBytes + r * 16);
        const bool whole = keys0 + 32 * kTiles - 1 <= p0 && (tile + 1) * kRowTile <= rows &&
                           (!c.a.window || keys0 > p1 - c.a.window);
        if (__builtin_expect(!whole, 0)) {
          const int row = tile * kRowTile + r;
          const int64_t pos = start + row / c.group;
          // of the keys counted from this half's first
          const int hi = row < rows ? (int)max(pos - keys0 - 4 * hf, (int64_t)-1) : -1;
          const int lo = c.a.window ? (int)max(pos - c.a.window + 1 - keys0 - 4 * hf, (int64_t)0) : 0;
#pragma unroll
          for (int u = 0; u < kTiles; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int key = 32 * u + 8 * (i / 4) + i % 4;
              const float w = weight_again(__builtin_fmaf(x[u][i], fk[u][i] * f.x, -f.y), c.cs, f.w) * f.z;
              sum[u][i] += key <= hi && key >= lo ? w : 0.0f;
            }
          continue;
        }
#pragma unroll
        for (int u = 0; u < kTiles; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sum[u][i] = __builtin_fmaf(weight_again(__builtin_fmaf(x[u][i], fk[u][i] * f.x, -f.y), c.cs, f.w), f.z,
                                       sum[u][i]);
      }
      // sums over the 32 columns; lane (r, hf) with r < 16 stores key r's register
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float w = sum[u][i];
          w += dpp_row_f<kDppQuadXor1>(w);
          w += dpp_row_f<kDppQuadXor2>(w);
          w += dpp_row_f<kDppRowRor4>(w);
          w += dpp_row_f<kDppRowRor8>(w);
          w += __shfl_xor(w, 16);
          // register i of half hf is key 8 (i / 4) + 4 hf + i % 4: to that key's lane
          const float other = __shfl_xor(w, 32);
          v = r == 8 * (i / 4) + i % 4 ? (hf ? other : w) : r == 8 * (i / 4) + 4 + i % 4 ? (hf ? w : other) : v;
        }
        const int key = keys0 + 32 * u + r;
        if (hf == 0 && ok[u] && key < len && (!c.a.window || key > start - c.a.window))
          add_weight(c.a.weights_out + at[u], v);
      }
    }
  }
}

unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20); }

template <int D>
hipError_t launch_d(const Call &c, hipStream_t s) {
  const int64_t rows = (int64_t)c.rows.tokens * c.a.q_heads;
  const hipError_t e = launch(kv_weight_rows_kernel<D>, dim3(grid_of((rows * (D / 8) + 255) / 256)), dim3(256), 0, s, c,
                              rows);
  if (e != hipSuccess) return e;
  const int64_t cap = (int64_t)c.rows.table_width << c.kv.shift, heads = (int64_t)c.rows.seqs * c.kv.p.kv_heads;
  // D = 256 has no registers for 64 keys a wave; elsewhere 32 where 64 leave CUs without a workgroup (two prompts of
  // 300 tokens on 2000 rows, 8 heads: 85 against 165 us).  At most four workgroups for every CU.
  constexpr int kMost = D == 256 ? 1 : 2;
  auto parts = [&](int keys) {
    const int64_t all = (cap + keys - 1) / keys, most = (1024 + heads - 1) / heads;
    return all < most ? all : most;
  };
  const int64_t many = heads * parts(kWaves * 32 * kMost), few = heads * parts(kWaves * 32);
  const bool small = c.kv.p.page_size == 16;
  if (many < 256)
    return launch(small ? kv_row_weights_kernel<D, 1, true> : kv_row_weights_kernel<D, 1, false>, dim3(grid_of(few)),
                  dim3(64 * kWaves), 0, s, c, few);
  return launch(small ? kv_row_weights_kernel<D, kMost, true> : kv_row_weights_kernel<D, kMost, false>,
                dim3(grid_of(many)), dim3(64 * kWaves), 0, s, c, many);
}

}  // namespace

hipError_t launch_row_weights(const Call &c, hipStream_t s) {
  switch (c.kv.p.head_dim) {
    case 64: return launch_d<64>(c, s);
    case 128: return launch_d<128>(c, s);
    default: return launch_d<256>(c, s);
  }
}

}  // namespace coli
