// Dense products with their epilogue (coli_moe_linear) for more than a few
// rows: out = act(x w^T [* sx sw] + bias) + residual.
//
// Bound by the matrix cores: 2 m n k operations on (m + n) k elements.  8192^3
// runs at 1.33 PFLOP/s in bf16 (the library's product: 1.49), 4096 x 6144 x
// 6144 at 1.12 (the library's: 1.12); there the chip is held by its power:
// the same call on zeros takes two thirds of the time, and reading every
// operand row from the L2 alone changes less.  4096 rows of 6144 int8 on 2048
// gate and 2048 up rows with SwiGLU run at 2.3 PFLOP/s; e4m3, on the 16-bit
// cores, at 1.29 for 8192^3 and 1.0 for 4096 x 6144 x 2048 onto a residual.  A
// workgroup computes a tile of BM x BN outputs over all of K in steps of 128
// bytes of every row (64 16-bit or 128 8-bit elements: one whole cache line a
// row).  Rows of x and w go straight into LDS by LDS-DMA, STAGES steps deep,
// 16-byte piece c of row r in position c ^ ((r >> 1) & 7), so that the 16
// rows that neighbouring lanes read fall into different banks.  Each wave
// holds MB x NB accumulators of 32 x 32; operands are read from LDS while
// others are multiplied, by the same wave (blocks of four waves) or by the
// other wave of its SIMD (blocks of eight).
//
// K that is not a multiple of the step: the pieces of the last step that lie
// past the rows' ends are copied from a piece of zeros.  Rows past the last
// of x or w: the last row again, results not stored.
//
// SwiGLU: w holds the n gate rows and then the n up rows.  A tile takes BN/2
// of each in alternating blocks of 32.  The gate and the up sum of an output
// meet in the epilogue's slab in LDS; a wave of one or three column blocks
// does not hold both.
//
// Blocks are mapped so that each XCD (hardware block b runs on XCD b mod 8)
// works on neighbouring tiles, 8 tiles high: the rows that they share come
// from that XCD's L2.
#include <type_traits>

#include "internal.h"
#include "linear.h"
#include "operators.h"

namespace coli {
namespace {

constexpr int kXcds = 8;
constexpr int kStepBytes = 128;  // of a row, per K step

template <int TYPE, int MB, int NB, int WM, int WN, int STAGES, bool GATED>
struct Tile {
  typedef Operand<TYPE> Op;
  typedef typename Op::Acc32 Acc;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int BM = 32 * MB * WM, BN = 32 * NB * WN;  // rows of x and of w
  static constexpr int kOutN = GATED ? BN / 2 : BN;           // output columns
  static constexpr int kStageBytes = (BM + BN) * kStepBytes;
  // the epilogue's slab: 32 rows of every wave row, padded so that the two
  // half-waves' rows (4 apart) fall into different banks
  static constexpr int kRowFloats = BN + 8;
  static constexpr int kEpilogueBytes = WM * 32 * kRowFloats * 4;
  static constexpr int kRing = STAGES * kStageBytes;
  static constexpr int kLds = kRing > kEpilogueBytes ? kRing : kEpilogueBytes;
  static_assert(kLds <= 160 * 1024, "the ring exceeds a CU's LDS");
  static_assert(BM / 8 % kWaves == 0 && BN / 8 % kWaves == 0, "copies of 8 rows, as many for each wave");
  static_assert(!GATED || BN % 64 == 0, "pairs of gate and up blocks");
  static constexpr int kCopiesA = BM / 8 / kWaves, kCopiesB = BN / 8 / kWaves, kCopies = kCopiesA + kCopiesB;

  // Where this lane's copies come from, relative to the tile's first rows.
  struct Sources {
    const char *x, *w, *up;  // tile's first row of x, of w (and of its up rows)
    uint32_t xo[kCopiesA], wo[kCopiesB];
    int64_t k_bytes;
  };

  // Copy i of a wave: rows 8 c .. 8 c + 7 of the tile's x or w rows, c = i
  // kWaves + wave; lane l copies position l % 8 of row 8 c + l / 8.
  static __device__ __forceinline__ uint32_t piece(int row, int lane) {
    return (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 16);
  }

  static __device__ __forceinline__ void copy_whole(const Sources &S, int i, int64_t at, uint32_t lds, int wave) {
    const bool a = i < kCopiesA;
    const int c = (a ? i : i - kCopiesA) * kWaves + wave;
    const char *base = a ? S.x : (GATED && (c & 4)) ? S.up : S.w;
    dma16(lds + (uint32_t)((a ? 0 : BM * kStepBytes) + c * 8 * kStepBytes), base + at,
          a ? S.xo[a ? i : 0] : S.wo[a ? 0 : i - kCopiesA]);
  }

  // The same for the last, partial step: pieces past K come from a piece of zeros.
  static __device__ __forceinline__ void copy_rest(const Sources &S, int i, int64_t at, uint32_t lds, int wave,
                                                   int lane) {
    const bool a = i < kCopiesA;
    const int c = (a ? i : i - kCopiesA) * kWaves + wave;
    const char *base = a ? S.x : (GATED && (c & 4)) ? S.up : S.w;
    const uint32_t off = a ? S.xo[a ? i : 0] : S.wo[a ? 0 : i - kCopiesA];
    const bool real = at + (int64_t)piece(8 * c + (lane >> 3), lane) < S.k_bytes;
    dma16v(lds + (uint32_t)((a ? 0 : BM * kStepBytes) + c * 8 * kStepBytes),
           real ? base + at + off : reinterpret_cast<const char *>(&kZeroPiece));
  }

  static __device__ __forceinline__ void run(const coli_moe_linear_t &a, char *lds_mem) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    // this block's tile
    const int tiles_n = (a.n + kOutN - 1) / kOutN, tiles_m = (a.m + BM - 1) / BM, tiles = tiles_m * tiles_n;
    const int b = blockIdx.x, xcd = b % kXcds;
    const int t = xcd * (tiles / kXcds) + min(xcd, tiles % kXcds) + b / kXcds;
    const int first = t / (kXcds * tiles_n) * kXcds, high = min(kXcds, tiles_m - first);
    const int in = t - first * tiles_n;
    const int m0 = (first + in % high) * BM, n0 = in / high * kOutN;

    constexpr size_t esz = TYPE == COLI_MOE_BF16 || TYPE == COLI_MOE_F16 ? 2 : 1;
    const size_t ldx = (size_t)a.ldx * esz, ldw = (size_t)a.ldw * esz;
    Sources S;
    S.x = static_cast<const char *>(a.x) + (size_t)m0 * ldx;
    S.w = static_cast<const char *>(a.w) + (size_t)n0 * ldw;
    S.up = S.w + (size_t)a.n * ldw;
    S.k_bytes = (int64_t)a.k * esz;
#pragma unroll
    for (int i = 0; i < kCopiesA; ++i) {
      const int row = 8 * (i * kWaves + wave) + (lane >> 3);
      S.xo[i] = (uint32_t)(min(row, a.m - 1 - m0) * ldx) + piece(row, lane);
    }
#pragma unroll
    for (int i = 0; i < kCopiesB; ++i) {
      const int row = 8 * (i * kWaves + wave) + (lane >> 3);
      const int col = GATED ? (row >> 6) * 32 + (row & 31) : row;  // output column of the row
      S.wo[i] = (uint32_t)(min(col, a.n - 1 - n0) * ldw) + piece(row, lane);
    }

    const uint32_t lds = lds_addr(lds_mem);
    const int G = (int)((S.k_bytes + kStepBytes - 1) / kStepBytes);
    Acc acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = Acc{};

    const int whole = (int)(S.k_bytes / kStepBytes);
    if (whole) {
      if constexpr (kWaves == 4)
        pipelined(S, whole, lds, lds_mem, wm, wn, wave, lane, acc);
      else if (wave >= 4)
        alternate<true>(S, whole, lds, lds_mem, wm, wn, wave, lane, acc);
      else
        alternate<false>(S, whole, lds, lds_mem, wm, wn, wave, lane, acc);
    }
    if (whole < G) remainder(S, whole, lds, lds_mem, wm, wn, wave, lane, acc);
    block_barrier();  // the ring is free
    epilogue(a, m0, n0, wm, wn, lane, acc, reinterpret_cast<float *>(lds_mem));
  }

  // Four waves, one on every SIMD: while a wave multiplies step g, it reads its
  // operands of step g + 1 into other registers, a few reads and copies after
  // each product, so that nothing waits for LDS.  Step g + 1 has arrived for
  // every wave at the barrier in front of step g; step g - 1's slot, whose
  // operands were in registers before step g - 1's products, takes step g +
  // STAGES - 1 from then on.  As in alternate, copies past the last step fetch
  // it again.  (256 x 6144 x 6144 bf16 in 128 x 64 blocks: 30 us; with the reads
  // in front of each step's products, also over six stages, 46 us; eight waves
  // taking turns 45 us; three stages, two blocks a CU, 59 us.  Reads spread over
  // all of a step's products, or within the first quarter, are as fast.)
  static __device__ __forceinline__ void pipelined(const Sources &S, int G, uint32_t lds, const char *lds_mem, int wm,
                                                   int wn, int wave, int lane, Acc (&acc)[MB][NB]) {
    constexpr int kAhead = STAGES - 1, kAll = 4 * MB * NB, kReads = 4 * (MB + NB);
    const int nl = lane & 31, half = lane >> 5, swz = (nl >> 1) & 7;
    const int at_a = (wm * MB * 32 + nl) * kStepBytes, at_b = (BM + wn * NB * 32 + nl) * kStepBytes;
    uint4 op[2][4][MB + NB];  // operands of this step and of the next, by piece: rows of w, then of x
    auto read = [&](const char *stage, int buf, int r) {
      const int p = r / (MB + NB), q = r % (MB + NB), pos = ((4 * half + p) ^ swz) * 16;
      op[buf][p][q] = *reinterpret_cast<const uint4 *>(
          stage + (q < NB ? at_b + q * 32 * kStepBytes : at_a + (q - NB) * 32 * kStepBytes) + pos);
    };
    auto copy_step = [&](int g, int slot, int i) {
      copy_whole(S, i, (int64_t)min(g, G - 1) * kStepBytes, lds + slot * kStageBytes, wave);
    };
    auto next = [](int slot) { return slot + 1 == STAGES ? 0 : slot + 1; };
#pragma unroll
    for (int g = 0; g < kAhead; ++g)
#pragma unroll
      for (int i = 0; i < kCopies; ++i) copy_step(g, g, i);
    dma_wait<kCopies *(STAGES - 2)>();
    turn();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(lds_mem, 0, r);
    int ahead = next(0), fill = kAhead;  // slots of step g + 1 and of step g + kAhead
    auto step = [&](int g, auto buf_) {
      constexpr int buf = decltype(buf_)::value;
      dma_wait<kCopies *(STAGES - 3)>();
      turn();
      const char *stage = lds_mem + ahead * kStageBytes;
#pragma unroll
      for (int j = 0; j < kAll; ++j) {
        const int p = j / (MB * NB), mb = j / NB % MB, nb = j % NB;
        acc[mb][nb] = Op::mma(op[buf][p][NB + mb], op[buf][p][nb], acc[mb][nb]);
#pragma unroll
        for (int r = kReads * min(2 * j, kAll) / kAll; r < kReads * min(2 * j + 2, kAll) / kAll; ++r)
          read(stage, buf ^ 1, r);
#pragma unroll
        for (int i = j * kCopies / kAll; i < (j + 1) * kCopies / kAll; ++i) copy_step(g + kAhead, fill, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      ahead = next(ahead);
      fill = next(fill);
    };
    int g = 0;
    for (; g + 1 < G; g += 2) {
      step(g, std::integral_constant<int, 0>());
      step(g + 1, std::integral_constant<int, 1>());
    }
    if (g < G) step(g, std::integral_constant<int, 0>());
    dma_wait<0>();
  }

  // Two groups of four waves, one of each on every SIMD, take turns: while one
  // group's waves multiply, the other's read their next operands, half a K
  // step, from LDS; a barrier ends each turn.  With the turns of step g
  // numbered 4 g .. 4 g + 3, the first group reads in turns 4 g and 4 g + 2
  // and multiplies in the other two; the second does the same one turn later.
  // Step g - 1's slot was last read in turn 4 g - 1 (second group), so step
  // g + STAGES - 1 is copied into it from turn 4 g on: half of a wave's copies
  // go out with the reads of the step's first half (turn 4 g or 4 g + 1), the
  // others between products, in turn 4 g + 1 (first group) and 4 g (second
  // group, with its last products of step g - 1).  Both groups await their
  // copies of step g + 1, those of later steps still going, before the barrier
  // that ends turn 4 g + 3, behind which turn 4 g + 4 reads them.  A third
  // stage pays where it fits beside one workgroup a CU (256 x 128: m = 1024 in
  // 82 us, with two 110).  (8192^3 bf16: 827 us; all copies with the reads 894
  // us, all between products 843 us; without the raised priority of the
  // multiplying waves 903 us.  4096 x 6144 x 6144 with bias and SiLU: 305 us a
  // call, 451 with every wave at its own pace, one barrier a step.)  The
  // copies have no conditions: past the last step they fetch it again, into
  // the slot that is not read any more (a branch a copy, between the products,
  // cost 23%).
  template <bool SECOND>
  static __device__ __forceinline__ void alternate(const Sources &S, int G, uint32_t lds, const char *lds_mem, int wm,
                                                   int wn, int wave, int lane, Acc (&acc)[MB][NB]) {
    constexpr int kAhead = STAGES - 1;    // steps between a copy and its use
    constexpr int kInRead = kCopies / 2;  // copies issued in a read turn, the others between products
    // copy i of step g into the slot that the ring gives it
    auto copy_step = [&](int g, int slot, int i) {
      copy_whole(S, i, (int64_t)min(g, G - 1) * kStepBytes, lds + slot * kStageBytes, wave);
    };
    auto next = [](int slot) { return slot + 1 == STAGES ? 0 : slot + 1; };
#pragma unroll
    for (int g = 0; g < kAhead; ++g)
#pragma unroll
      for (int i = 0; i < kCopies; ++i) copy_step(g, g, i);
    dma_wait<kCopies *(STAGES - 2)>();
    turn();
    if (SECOND) {
#pragma unroll
      for (int i = kInRead; i < kCopies; ++i) copy_step(kAhead, kAhead, i);
      turn();
    }
    int slot = 0, fill = kAhead;  // slots of step g and of step g + kAhead
    for (int g = 0; g < G; ++g) {
      if constexpr (STAGES == 2) {
        slot = g & 1;
        fill = slot ^ 1;
      }
      const char *stage = lds_mem + slot * kStageBytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 af[MB][2], bf[NB][2];
        fetch_half(stage, wm, wn, lane, h, af, bf);
        if (h == 0)
#pragma unroll
          for (int i = 0; i < kInRead; ++i) copy_step(g + kAhead, fill, i);
        if (h == 1 && SECOND) dma_wait<kCopies *(STAGES - 2)>();
        lds_wait();
        turn();
        __builtin_amdgcn_s_setprio(1);
        multiply_half(af, bf, acc, [&](int i) {
          if (SECOND == (h == 1) && i >= kInRead)
            copy_step(g + kAhead + h, h ? (STAGES == 2 ? slot : next(fill)) : fill, i);
        });
        __builtin_amdgcn_s_setprio(0);
        if (h == 1 && !SECOND) dma_wait<kCopies *(STAGES - 2)>();
        turn();
      }
      slot = next(slot);
      fill = next(fill);
    }
    if (!SECOND) turn();
    dma_wait<0>();
  }

  // The last step of a K that is no multiple of it.
  static __device__ __forceinline__ void remainder(const Sources &S, int G, uint32_t lds, const char *lds_mem, int wm,
                                                   int wn, int wave, int lane, Acc (&acc)[MB][NB]) {
    block_barrier();
#pragma unroll
    for (int i = 0; i < kCopies; ++i) copy_rest(S, i, (int64_t)G * kStepBytes, lds, wave, lane);
    dma_wait<0>();
    block_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 af[MB][2], bf[NB][2];
      fetch_half(lds_mem, wm, wn, lane, h, af, bf);
      multiply_half(af, bf, acc, [](int) {});
    }
  }

  static __device__ __forceinline__ void turn() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }
  static __device__ __forceinline__ void lds_wait() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  // This lane's operands of half h of a step: 2 pieces of each of its rows.
  static __device__ __forceinline__ void fetch_half(const char *stage, int wm, int wn, int lane, int h,
                                                    uint4 (&af)[MB][2], uint4 (&bf)[NB][2]) {
    const int nl = lane & 31, half = lane >> 5, swz = (nl >> 1) & 7;
    const char *A = stage + (wm * MB * 32 + nl) * kStepBytes;
    const char *B = stage + (BM + wn * NB * 32 + nl) * kStepBytes;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int pos = ((4 * half + 2 * h + p) ^ swz) * 16;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) bf[nb][p] = *reinterpret_cast<const uint4 *>(B + nb * 32 * kStepBytes + pos);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) af[mb][p] = *reinterpret_cast<const uint4 *>(A + mb * 32 * kStepBytes + pos);
    }
  }

  // The products of half a step, copy i of the wave's kCopies issued after an
  // equal share of them.
  template <class Copy>
  static __device__ __forceinline__ void multiply_half(const uint4 (&af)[MB][2], const uint4 (&bf)[NB][2],
                                                       Acc (&acc)[MB][NB], const Copy &copy_one) {
    constexpr int kAll = 2 * MB * NB;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          acc[mb][nb] = Op::mma(af[mb][p], bf[nb][p], acc[mb][nb]);
          const int done = (p * MB + mb) * NB + nb;
#pragma unroll
          for (int i = done * kCopies / kAll; i < (done + 1) * kCopies / kAll; ++i) copy_one(i);
        }
  }

  // Accumulators -> LDS -> 8 neighbouring outputs a thread, a slab of 32 rows
  // of every wave row at a time.  Register i of a 32 x 32 block is row
  // 8 (i / 4) + 4 half + i % 4, the lane's column is lane % 32.  The loop over
  // the slabs stays a loop (only the accumulators' registers differ), and
  // tiles that end inside 8 columns take their own copy of the code: it runs
  // once a tile, straight from memory.
  static __device__ __forceinline__ void epilogue(const coli_moe_linear_t &a, int m0, int n0, int wm, int wn, int lane,
                                                  const Acc (&acc)[MB][NB], float *sums) {
    const int nl = lane & 31, half = lane >> 5;
    const bool whole = n0 + kOutN <= a.n;
#pragma nounroll
    for (int mb = 0; mb < MB; ++mb) {
      if (mb) __syncthreads();
      float *to = sums + (wm * 32 + 4 * half) * kRowFloats + 32 * wn * NB + nl;
#pragma unroll
      for (int q = 0; q < MB; ++q)
        if (q == mb) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 16; ++i) to[(8 * (i >> 2) + (i & 3)) * kRowFloats + 32 * nb] = (float)acc[q][nb][i];
        }
      __syncthreads();
      if (whole)
        finish_slab<true>(a, m0, n0, mb, sums);
      else
        finish_slab<false>(a, m0, n0, mb, sums);
    }
  }

  // One slab: scales, bias and activation in LDS (a loop: one copy of that
  // code), then residual and store; every residual of the slab is on its way
  // before that.  Each thread stays with its own outputs.
  template <bool WHOLE>
  static __device__ __forceinline__ void finish_slab(const coli_moe_linear_t &a, int m0, int n0, int mb, float *sums) {
    constexpr int kParts = kOutN / 8, kTurns = WM * 32 * kParts / kThreads;
    static_assert(kTurns * kThreads == WM * 32 * kParts, "whole turns of the threads");
    // The slabs' loop leaves each thread's columns alone, and the compiler would
    // compute every address of every turn ahead of it and keep them all (100
    // registers, of which other workgroups of the CU have no use); an index
    // that it cannot see through keeps them in the loop.
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    auto row = [&](int i) {
      const int r = (tid + i * kThreads) / kParts;
      return m0 + ((r >> 5) * MB + mb) * 32 + (r & 31);
    };
    auto column = [&](int i) { return n0 + (tid + i * kThreads) % kParts * 8; };
    auto place = [&](int i) {
      const int q = tid + i * kThreads, r = q / kParts, c = q % kParts * 8;
      return sums + r * kRowFloats + (GATED ? (c >> 5) * 64 + (c & 31) : c);
    };
    Raw8 res[kTurns];
    if (WHOLE && a.residual) {  // rows past the last read the last
      if (a.out_type == COLI_MOE_F32) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i)
          res[i] = load_raw8(a.residual, COLI_MOE_F32, (int64_t)min(row(i), a.m - 1) * a.ldr + column(i));
      } else {
#pragma unroll
        for (int i = 0; i < kTurns; ++i)
          res[i] = load_raw8(a.residual, COLI_MOE_BF16, (int64_t)min(row(i), a.m - 1) * a.ldr + column(i));
      }
    }
    float v[8], up[8];
    if (a.x_scale || a.bias || a.act != COLI_MOE_ACT_NONE) {
#pragma nounroll
      for (int i = 0; i < kTurns; ++i) {
        if (row(i) >= a.m || column(i) >= a.n) continue;
        float *at = place(i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = at[j];
          up[j] = GATED ? at[32 + j] : 0.0f;
        }
        activate8<WHOLE>(a, row(i), column(i), v, up);
#pragma unroll
        for (int j = 0; j < 8; ++j) at[j] = v[j];
      }
    }
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      if (row(i) >= a.m || column(i) >= a.n) continue;
      const float *at = place(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = at[j];
      if (!WHOLE && a.residual)
        res[i] = load_raw8(a.residual, a.out_type, (int64_t)row(i) * a.ldr + column(i), a.n - column(i));
      store_out8<WHOLE>(a, row(i), column(i), v, res[i]);
    }
  }
};

// One workgroup a CU, by its LDS: one or two waves on each SIMD share its registers.
template <class T>
__global__ __launch_bounds__(T::kThreads, T::kWaves / 4) void linear_tile_kernel(coli_moe_linear_t a) {
  __shared__ __attribute__((aligned(16))) char lds[T::kLds];
  T::run(a, lds);
}

template <int TYPE, int MB, int NB, int WM, int WN, int STAGES>
hipError_t launch_tiles(const coli_moe_linear_t &a, hipStream_t s) {
  auto go = [&](auto gated) -> hipError_t {
    typedef Tile<TYPE, MB, NB, WM, WN, STAGES, decltype(gated)::value> T;
    const int64_t tiles = (int64_t)((a.m + T::BM - 1) / T::BM) * ((a.n + T::kOutN - 1) / T::kOutN);
    return launch(linear_tile_kernel<T>, dim3((uint32_t)tiles), dim3(T::kThreads), 0, s, a);
  };
  return a.act == COLI_MOE_ACT_SWIGLU ? go(std::true_type()) : go(std::false_type());
}

// The shapes a product of more than kLinearRowsMax rows can take, one block a
// CU, with what they cost: microseconds measured at 12288 bytes of K (6144
// bf16 elements; n = 6144, m from 64 to 4096, three sets of operands in turn)
// for up to one block a CU, and for a round that fills the chip (the clock
// held by the power).  The same costs rank the shapes for every type and K,
// though int8 takes half the matrix time and a short K is ruled by what a
// block costs beside its steps: neither was fitted.
struct Shape {
  int bm, bn;     // rows of x and of w of a block
  int one, full;  // cost of a round with fewer blocks, and of a full one
};
constexpr int kCus = 256;
constexpr Shape kShapes[] = {
    {64, 32, 17, 17},      // linear_rows: m = 64 in 18 to 20 us, 128 in 34, 256 in 50
    {64, 64, 21, 25},      // four waves: m = 128 in 21 us, 256 (384 blocks) in 41, 512 (three full rounds) in 81
    {128, 64, 30, 38},     // the same: m = 256 in 30 us, 512 (384 blocks) in 62, 1024 (three full rounds) in 124
    {128, 128, 48, 57},    // the same: m = 384 in 39 us, 512 in 46 to 58, 640 in 60, 1024 (384 blocks) in 115
    {256, 128, 84, 91},    // eight waves: m = 1024 in 82 us (192 blocks), 4096 in 273 (three full rounds)
    {256, 192, 136, 136},  // m = 2048 in 140 us, 4096 in 272 (two full rounds)
    {256, 256, 150, 150},  // m = 2048 in 152 us, 4096 in 296 (two rounds, the second half empty)
};

// The shape with the least cost: rounds of blocks over the CUs times the
// cost of a round.  Large blocks read less per product, small ones leave
// fewer CUs idle.
int pick_shape(int64_t m, int64_t wrows) {
  int best = 0;
  int64_t least = 0;
  for (int i = 0; i < (int)(sizeof(kShapes) / sizeof(kShapes[0])); ++i) {
    const Shape &s = kShapes[i];
    const int64_t blocks = ((m + s.bm - 1) / s.bm) * ((wrows + s.bn - 1) / s.bn);
    const int64_t cost = blocks / kCus * s.full + (blocks % kCus ? s.one : 0);
    if (i == 0 || cost < least) {
      best = i;
      least = cost;
    }
  }
  return best;
}

template <int TYPE>
hipError_t launch_type(const coli_moe_linear_t &a, int shape, hipStream_t s) {
  switch (shape) {
    case 1: return launch_tiles<TYPE, 1, 1, 2, 2, 8>(a, s);
    case 2: return launch_tiles<TYPE, 2, 1, 2, 2, 6>(a, s);
    case 3: return launch_tiles<TYPE, 2, 2, 2, 2, 4>(a, s);
    case 4: return launch_tiles<TYPE, 2, 2, 4, 2, 3>(a, s);
    case 5: return launch_tiles<TYPE, 2, 3, 4, 2, 2>(a, s);
    default: return launch_tiles<TYPE, 4, 2, 2, 4, 2>(a, s);
  }
}

}  // namespace

hipError_t launch_linear(const coli_moe_linear_t &a, hipStream_t s) {
  if (a.m <= kLinearRowsMax) return launch_linear_rows(a, s);
  const int shape = pick_shape(a.m, a.act == COLI_MOE_ACT_SWIGLU ? 2 * (int64_t)a.n : a.n);
  if (shape == 0) return launch_linear_rows(a, s);
  switch (a.type) {
    case COLI_MOE_BF16: return launch_type<COLI_MOE_BF16>(a, shape, s);
    case COLI_MOE_F16: return launch_type<COLI_MOE_F16>(a, shape, s);
    case COLI_MOE_INT8: return launch_type<COLI_MOE_INT8>(a, shape, s);
    default: return launch_type<COLI_MOE_E4M3>(a, shape, s);
  }
}

}  // namespace coli
