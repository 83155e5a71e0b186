// Dense products with their epilogue (coli_moe_linear) for few rows of x
// (up to kLinearRowsMax): decode steps and small batches.
//
// Bound by the bytes of w, each read once (beyond kLinearRowsMax rows, where
// few large blocks would leave most CUs idle: once per 64 rows of x).  A
// workgroup owns 16 or 32 rows of w (SwiGLU: half of them gate rows, half
// the up rows of the same outputs) and splits K over its four waves: each wave
// takes every fourth chunk of CB bytes of every row, copies it with the
// matching chunk of x into its own ring of 2 or 3 slots in LDS by LDS-DMA, and
// multiplies it on 16x16 matrix instructions (16 rows of w by 16 rows of x).
// Up to 32 rows of x a chunk is long (256 or 512 bytes of a row), because
// short pieces of rows read HBM poorly; it goes through LDS because the
// instructions want 16 rows by 64 bytes.  The waves never wait for each other
// before the end, where their sums meet in LDS in wave order.
//
// The 16-byte pieces of a row change places with the row (swizzle below), so
// that the 16 rows that neighbouring lanes read fall into different banks.
// Rows past the last of x or w: the last row again, results not stored.
// Pieces past K come from a piece of zeros.
#include <type_traits>

#include "internal.h"
#include "linear.h"
#include "operators.h"

namespace coli {
namespace {

constexpr int kWaves = 4;
constexpr int kXcds = 8;

// MR: rows of x a workgroup holds (a power of two); RT: 16-row tiles of w it
// owns; CB: bytes of a chunk.
template <int TYPE, int MR, int RT, int CB, int SLOTS, bool GATED>
struct Rows {
  typedef Operand<TYPE> Op;
  typedef typename Op::Acc16 Acc;
  typedef std::conditional_t<TYPE == COLI_MOE_INT8, int, float> Sum;
  static constexpr int WR = 16 * RT;              // rows of w
  static constexpr int kRowsPerCopy = 1024 / CB;  // rows of one wave's copy (64 lanes x 16 bytes)
  static constexpr int kCopiesW = WR / kRowsPerCopy, kCopiesX = MR / kRowsPerCopy, kCopies = kCopiesW + kCopiesX;
  static constexpr int kTokens = MR <= 16 ? 1 : MR / 16;  // 16-row tiles of x
  static constexpr int kSlotBytes = (WR + MR) * CB;
  static constexpr int kWaveBytes = SLOTS * kSlotBytes;
  static constexpr int kOutN = GATED ? WR / 2 : WR;
  static_assert(kCopiesX >= 1 && kWaves * kWaveBytes <= 160 * 1024, "ring");
  static_assert(kTokens * RT * 256 * 4 <= kWaveBytes, "the sums take the ring's place");

  // What a piece's position is xored with: 16 rows that neighbouring lanes
  // read at the same piece fall into different banks (64 banks: two rows of
  // 128 bytes, or one of 256 and more).
  static __device__ __forceinline__ int swizzle(int row) { return CB >= 256 ? row & 15 : (row >> 1) & 7; }

  // Chunk c of this wave has arrived once at most the copies of its later
  // chunks (up to LATER of them) are pending.
  template <int LATER>
  static __device__ __forceinline__ void wait_for(int c, int chunks) {
    if constexpr (LATER > 0) {
      if (c + LATER * kWaves >= chunks) {
        wait_for<LATER - 1>(c, chunks);
        return;
      }
    }
    dma_wait<LATER * kCopies>();
  }

  static __device__ __forceinline__ void run(const coli_moe_linear_t &a, char *lds_mem) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    // hardware block b runs on XCD b mod 8; an XCD gets a run of neighbouring
    // blocks, those of the same rows of w first
    const int blocks_m = (a.m + MR - 1) / MR, blocks = gridDim.x, xcd = blockIdx.x % kXcds;
    const int b = xcd * (blocks / kXcds) + min(xcd, blocks % kXcds) + blockIdx.x / kXcds;
    const int n0 = b / blocks_m * kOutN, m0 = b % blocks_m * MR;
    constexpr size_t esz = TYPE == COLI_MOE_BF16 || TYPE == COLI_MOE_F16 ? 2 : 1;
    const size_t ldx = (size_t)a.ldx * esz, ldw = (size_t)a.ldw * esz;
    const char *x = static_cast<const char *>(a.x) + (size_t)m0 * ldx;
    const char *w = static_cast<const char *>(a.w) + (size_t)n0 * ldw, *up = w + (size_t)a.n * ldw;
    const int64_t k_bytes = (int64_t)a.k * esz;
    const int chunks = (int)((k_bytes + CB - 1) / CB);
    char *mine = lds_mem + wave * kWaveBytes;
    const uint32_t lds = lds_addr(mine);

    // lane l copies position l % (CB / 16) of row l / (CB / 16) of each copy
    constexpr int kPer = CB / 16;
    const int at = lane % kPer, sub = lane / kPer;
    uint32_t wo[kCopiesW], xo[kCopiesX];
#pragma unroll
    for (int i = 0; i < kCopiesW; ++i) {
      const int row = i * kRowsPerCopy + sub, out = GATED ? row % kOutN : row;
      wo[i] = (uint32_t)(min(out, a.n - 1 - n0) * ldw) + (uint32_t)((at ^ swizzle(row)) * 16);
    }
#pragma unroll
    for (int i = 0; i < kCopiesX; ++i) {
      const int row = i * kRowsPerCopy + sub;
      xo[i] = (uint32_t)(min(row, a.m - 1 - m0) * ldx) + (uint32_t)((at ^ swizzle(row)) * 16);
    }
    auto issue = [&](int c, int slot) {
      const int64_t k0 = (int64_t)c * CB;
      const bool whole = k0 + CB <= k_bytes;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const bool is_x = i < kCopiesX;
        const int j = is_x ? i : i - kCopiesX;
        const char *base = is_x ? x : GATED && j >= kCopiesW / 2 ? up : w;
        const uint32_t off = is_x ? xo[is_x ? j : 0] : wo[is_x ? 0 : j];
        const uint32_t to = lds + (uint32_t)(slot * kSlotBytes + (is_x ? WR * CB : 0) + j * 1024);
        if (whole) {
          dma16(to, base + k0, off);
        } else {
          const int row = j * kRowsPerCopy + sub;
          const bool real = k0 + ((at ^ swizzle(row)) * 16) < k_bytes;
          dma16v(to, real ? base + k0 + off : reinterpret_cast<const char *>(&kZeroPiece));
        }
      }
    };

    Acc acc[RT][kTokens];
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int t = 0; t < kTokens; ++t) acc[q][t] = Acc{};
    // with fewer than 16 rows of x, the lanes of the missing ones read row
    // r mod MR: their columns of the result are not used
    const int r = lane & 15, g = lane >> 4, rx = r % MR;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
      if (wave + s * kWaves < chunks) issue(wave + s * kWaves, s);
    int slot = 0;
    for (int c = wave; c < chunks; c += kWaves) {
      wait_for<SLOTS - 1>(c, chunks);
      const char *W = mine + slot * kSlotBytes + r * CB, *X = mine + slot * kSlotBytes + WR * CB + rx * CB;
#pragma unroll
      for (int j = 0; j < CB / 64; ++j) {
        const int pw = ((4 * j + g) ^ swizzle(r)) * 16, px = ((4 * j + g) ^ swizzle(rx)) * 16;
        uint4 wf[RT];
#pragma unroll
        for (int q = 0; q < RT; ++q) wf[q] = *reinterpret_cast<const uint4 *>(W + q * 16 * CB + pw);
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
          const uint4 xf = *reinterpret_cast<const uint4 *>(X + t * 16 * CB + px);
#pragma unroll
          for (int q = 0; q < RT; ++q) acc[q][t] = Op::mma(wf[q], xf, acc[q][t]);
        }
      }
      // the slot's reads are done before it is copied to again
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (c + SLOTS * kWaves < chunks) issue(c + SLOTS * kWaves, slot);
      slot = slot + 1 == SLOTS ? 0 : slot + 1;
    }

    // the waves' sums, then the epilogue of 8 outputs a thread; register i of
    // lane l is row 4 (l / 16) + i of w and row l % 16 of x
    Sum *sums = reinterpret_cast<Sum *>(mine);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int t = 0; t < kTokens; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[(16 * t + r) * WR + 16 * q + 4 * g + i] = acc[q][t][i];
    __syncthreads();
    constexpr int kParts = kOutN / 8;
    for (int i = threadIdx.x; i < MR * kParts; i += 64 * kWaves) {
      const int token = i / kParts, part = i % kParts * 8;
      if (m0 + token >= a.m) break;
      if (n0 + part >= a.n) continue;
      Raw8 res;
      if (a.residual)
        res = load_raw8(a.residual, a.out_type, (int64_t)(m0 + token) * a.ldr + n0 + part, a.n - n0 - part);
      float v[8], u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        Sum s = 0, su = 0;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) {
          const Sum *p = reinterpret_cast<const Sum *>(lds_mem + q * kWaveBytes) + token * WR + part + e;
          s += p[0];
          if (GATED) su += p[kOutN];
        }
        v[e] = (float)s;
        u[e] = (float)su;
      }
      activate8<false>(a, m0 + token, n0 + part, v, u);
      store_out8<false>(a, m0 + token, n0 + part, v, res);
    }
  }
};

template <class T>
__global__ __launch_bounds__(64 * kWaves) void linear_rows_kernel(coli_moe_linear_t a) {
  __shared__ __attribute__((aligned(16))) char lds[kWaves * T::kWaveBytes];
  T::run(a, lds);
}

template <int TYPE, int MR, int RT, int CB, int SLOTS>
hipError_t launch_shape(const coli_moe_linear_t &a, hipStream_t s) {
  auto go = [&](auto gated) {
    typedef Rows<TYPE, MR, RT, CB, SLOTS, decltype(gated)::value> R;
    const int64_t blocks = (int64_t)((a.n + R::kOutN - 1) / R::kOutN) * ((a.m + MR - 1) / MR);
    return launch(linear_rows_kernel<R>, dim3((uint32_t)blocks), dim3(64 * kWaves), 0, s, a);
  };
  return a.act == COLI_MOE_ACT_SWIGLU ? go(std::true_type()) : go(std::false_type());
}

// Up to 16 rows of x, LDS is kept small enough for two workgroups a CU: 16
// rows of bf16 on 6144 x 6144 take 13.9 us with 256-byte chunks (64 KB) and
// 17.0 us with 512-byte ones (128 KB), one row 12.9 us against 14.5 us with a
// third slot.  From 17 rows on, 32 rows of w share each chunk of x: 32 rows
// take 16.2 us, 18.9 us with 16 rows of w.
template <int TYPE>
hipError_t launch_type(const coli_moe_linear_t &a, hipStream_t s) {
  if (a.m <= 2) return launch_shape<TYPE, 2, 1, 512, 2>(a, s);
  if (a.m <= 4) return launch_shape<TYPE, 4, 1, 512, 2>(a, s);
  if (a.m <= 8) return launch_shape<TYPE, 8, 1, 256, 3>(a, s);
  if (a.m <= 16) return launch_shape<TYPE, 16, 1, 256, 2>(a, s);
  if (a.m <= 32) return launch_shape<TYPE, 32, 2, 256, 2>(a, s);
  return launch_shape<TYPE, 64, 2, 128, 2>(a, s);
}

}  // namespace

hipError_t launch_linear_rows(const coli_moe_linear_t &a, hipStream_t s) {
  switch (a.type) {
    case COLI_MOE_BF16: return launch_type<COLI_MOE_BF16>(a, s);
    case COLI_MOE_F16: return launch_type<COLI_MOE_F16>(a, s);
    case COLI_MOE_INT8: return launch_type<COLI_MOE_INT8>(a, s);
    default: return launch_type<COLI_MOE_E4M3>(a, s);
  }
}

}  // namespace coli
