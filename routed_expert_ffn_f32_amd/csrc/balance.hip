// Balance loss of the router's choices and its gradient with respect to the
// router's logits (coli_moe_balance, coli_moe_balance_grad).
//
// With each valid token's shares p_te of its logits (softmax, or sigmoid
// scores over their sum) and the kept assignments n_e of a sequence:
//   loss = alpha sum_e (E n_e / N) (1/V) sum_t p_te
//   coef_e = (alpha / V) (E n_e / N - 1)
//   d_te = dloss (coef_e - sum_j coef_j p_tj) p_te                        softmax
//   d_te = dloss (coef_e - sum_j coef_j p_tj) s_te (1 - s_te) / sum_j s_tj  sigmoid
//
// Bound by bytes: the loss reads logits and choices once, the gradient reads
// the logits once and writes as much.  One wave takes a token, expert e in
// lane e mod 64, so a row's sums are wave reductions; four tokens at a time
// give the loads and the reductions something to overlap with.  Sigmoid over
// 256 experts: 65536 tokens take 24 us for the sums and 28 us for the gradient
// from HBM (2.8 and 4.8 TB/s), 19 and 23 us from the 256 MB cache; 16384
// tokens in 8 sequences 10, 5 (the joining launch) and 11 us.  There a
// workgroup of the sums has one batch of 64 tokens, whose loads, scores,
// reductions and join in LDS run one after another; a second batch, loaded
// meanwhile, adds 3.7 us (4.8 TB/s).
//
// Sums over tokens: a workgroup owns a run of consecutive tokens (a chunk)
// and visits the pieces of sequences in it.  A piece's sums go to slot
// (chunk + sequence) of the workspace: going through the tokens in order,
// each next piece has a larger chunk, a larger sequence, or both, so no two
// pieces share a slot.  A second launch adds a sequence's pieces in float64
// in a fixed order.  No atomics on floats: the same call gives the same bits.
#include "internal.h"
#include "wave.h"

#include <algorithm>
#include <type_traits>

#include "coli_moe.h"
#include "operators.h"
#include "scalar_math.h"

namespace coli {
namespace {

constexpr int kTok = 4;              // tokens a wave works on at once
constexpr int kSumWaves = 16;        // waves of a workgroup of the sums
constexpr int kSumThreads = 64 * kSumWaves;
constexpr int kMaxChunks = 256;      // workgroups of the sums, up to 2^20 tokens: one a CU (of two a CU, at
                                     // half the registers, 65536 tokens take 43 us against 24)
constexpr int kBatchTokens = kTok * kSumWaves;  // tokens they take at a time
constexpr int kAloneSeqs = 8;        // sequences of one batch that its workgroup finishes itself, one by one
constexpr int kGradWaves = 4;        // waves of a workgroup of the gradient, four tokens each

// A token's scores: v = exp(z - max) (softmax) or sigma(z), slope = its own
// derivative (softmax: v again), total their sum over the experts.
template <int NE, bool SOFTMAX>
struct Scores {
  float v[NE], slope[NE], total;
};

template <int NE, bool SOFTMAX>
__device__ __forceinline__ void score_tokens(const float (&z)[kTok][NE], int lane, int E,
                                             Scores<NE, SOFTMAX> (&out)[kTok]) {
  float top[kTok];
  if constexpr (SOFTMAX) {
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      float m = z[t][0];
#pragma unroll
      for (int i = 1; i < NE; ++i) m = fmaxf(m, z[t][i]);
      top[t] = m;
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t) top[t] = lanes_max<64>(top[t]);
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      float v, d;
      if constexpr (SOFTMAX) {
        // all -Inf: nothing to subtract, every share 0 (a NaN, which the
        // maximum leaves out, stays one)
        v = z[t][i] == -__builtin_inff() ? 0.0f : exp_neg(z[t][i] - top[t]);
        d = v;
      } else {
        // a = exp(-|z|): sigma and sigma (1 - sigma) = a / (1 + a)^2 without
        // overflow or cancellation
        const float a = exp_neg(-fabsf(z[t][i]));
        const float q = __builtin_amdgcn_rcpf(1.0f + a);
        v = (z[t][i] >= 0.0f ? 1.0f : a) * q;
        d = a * q * q;
      }
      const bool real = lane + 64 * i < E;
      out[t].v[i] = real ? v : 0.0f;
      out[t].slope[i] = real ? d : 0.0f;
      sum += out[t].v[i];
    }
    out[t].total = sum;
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t) out[t].total = wave_sum(out[t].total);
}

// Offsets clamped to the tokens.
__device__ __forceinline__ int seq_at(const coli_moe_balance_t &a, int s) {
  if (!a.seq_offsets) return s == 0 ? 0 : a.tokens;
  return min(max(a.seq_offsets[s], 0), a.tokens);
}

// The sequences' bounds, 64 at a time in the wave's lanes (a load for each
// bound would be a memory round trip in front of everything else).
struct Bounds {
  int first, value;  // lane l holds the start of sequence first + l

  __device__ __forceinline__ void load(const coli_moe_balance_t &a, int s) {
    first = s;
    value = seq_at(a, min(s + (int)(threadIdx.x & 63), a.n_seqs));
  }
  // Start and end of sequence s < n_seqs, s >= first.  A window without the
  // end is moved to start at s itself, never behind it: the caller may ask for
  // s again, for the tokens of its next batch.
  __device__ __forceinline__ void of(const coli_moe_balance_t &a, int s, int &begin, int &end) {
    if (s + 1 - first >= 64) load(a, s);
    begin = __builtin_amdgcn_readlane(value, s - first);
    end = __builtin_amdgcn_readlane(value, s + 1 - first);
  }
  // Starts at the first sequence that ends behind token t (n_seqs: none):
  // the number of ends at or before t, narrowed 64-fold a load.  For up to 63
  // sequences load(a, 0), issued earlier, is all it needs.
  __device__ __forceinline__ int seek(const coli_moe_balance_t &a, int t) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = a.n_seqs;  // among sequences lo .. lo + n - 1 or behind them
    if (n > 63) {
      do {
        const int step = (n + 62) / 63, probe = min(lo + step * (lane + 1), lo + n);
        const int before = __popcll(__ballot(seq_at(a, probe) <= t));  // probes are ends, ascending
        const int skip = min(before * step, n);
        lo += skip;
        n = min(step, n - skip);
      } while (n > 63);
      load(a, lo);
    }
    return lo + __popcll(__ballot(lane >= 1 && lane <= n && value <= t));
  }
};

// A wave's next four tokens, t0 + t step: logits and mask as they stand.
// Masked tokens' logits are loaded (beside the mask, not behind it) but not
// looked at.
template <int NE>
struct Tokens {
  float raw[kTok][NE];
  uint8_t valid[kTok];

  __device__ __forceinline__ void load(const coli_moe_balance_t &a, int t0, int step, int end, int lane) {
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      const int tok = min(t0 + t * step, end - 1);
      valid[t] = a.mask ? a.mask[tok] : 1;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        raw[t][i] = a.logits[(int64_t)tok * a.logits_stride + min(lane + 64 * i, a.n_experts - 1)];
    }
  }
  __device__ __forceinline__ void look(int t0, int step, int end, int lane, int E, float (&z)[kTok][NE],
                                       bool (&on)[kTok]) const {
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      on[t] = t0 + t * step < end && valid[t] != 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) z[t][i] = on[t] && lane + 64 * i < E ? raw[t][i] : -__builtin_inff();
    }
  }
};

// Sums of one piece: share sums [E], counts [E], valid tokens (as float32
// words: E floats, then E + 1 ints).
__host__ __device__ inline size_t slot_words(int E) { return 2 * (size_t)E + 1; }

// What the sums of a sequence give: V valid tokens, N kept assignments, dot =
// sum_e n_e sum_t p_te, and thread `col`'s own count c.
__device__ __forceinline__ void finish_sequence(const coli_moe_balance_t &a, int s, int col, bool mine, int c, double V,
                                                double N, double dot, float *loss, int32_t *counts, float *coef) {
  const bool some = V > 0.0 && N > 0.0;
  const double per_token = some ? (double)a.alpha / V : 0.0, share = some ? a.n_experts / N : 0.0;
  if (threadIdx.x == 0) loss[s] = (float)(per_token * share * dot);
  if (mine) {
    counts[(size_t)s * a.n_experts + col] = c;
    coef[(size_t)s * a.n_experts + col] = (float)(per_token * ((double)c * share - 1.0));
  }
}

// Totals of N values over a workgroup of 1024 threads, in every thread.
template <int N>
__device__ __forceinline__ void block_totals(double (&v)[N], double (*scratch)[16]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lanes_sum64<64>(v[i]);
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) scratch[i][threadIdx.x >> 6] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.0;
#pragma unroll
    for (int w = 0; w < 16; ++w) v[i] += scratch[i][w];
  }
}

// A workgroup takes its tokens 64 at a time, four a wave; their loads need no
// knowledge of the sequences and go out first.  A piece's sums stay in
// registers (shares) and LDS (counts) until the piece ends.  ALONE: one
// workgroup and one batch hold every token, so each piece is a whole sequence
// and is finished on the spot (64 tokens: one launch of 5.6 us instead of two
// of 5.0 and 3.9 us and the gap between them).
template <int NE, bool SOFTMAX, bool ALONE>
__global__ __launch_bounds__(kSumThreads) void balance_sums_kernel(coli_moe_balance_t a, int chunk_tokens, float *slots,
                                                                   float *loss, int32_t *counts, float *coef) {
  __shared__ double totals[2][16];
  constexpr int kBatch = kBatchTokens, kIdx = kBatch * kMaxTopK / kSumThreads;
  __shared__ float mass[kSumWaves][64 * NE];
  __shared__ int hist[64 * NE];
  __shared__ int valid;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), E = a.n_experts, k = a.top_k;
  const int lo = blockIdx.x * chunk_tokens, hi = min(lo + chunk_tokens, a.tokens);
  Tokens<NE> now;
  int expert[kIdx], of[kIdx];  // this thread's assignments of the batch and their tokens
  uint8_t counted[kIdx];       // whether those tokens are valid
  auto load = [&](int t0) {
    now.load(a, t0 + wave, kSumWaves, hi, lane);
#pragma unroll
    for (int q = 0; q < kIdx; ++q) {
      const int i = threadIdx.x + q * kSumThreads;
      of[q] = t0 + (int)((uint32_t)i / (uint32_t)k);
      of[q] = i < kBatch * k && of[q] < hi ? of[q] : -1;
      expert[q] = of[q] >= 0 ? a.idx[(int64_t)t0 * k + i] : -1;
      counted[q] = a.mask && of[q] >= 0 ? a.mask[of[q]] : 1;
    }
  };
  Bounds bounds;
  bounds.load(a, 0);
  load(lo);
  int s = ALONE ? 0 : bounds.seek(a, lo);
  for (int i = threadIdx.x; i < E; i += kSumThreads) hist[i] = 0;
  if (threadIdx.x == 0) valid = 0;
  __syncthreads();
  float acc[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) acc[i] = 0.0f;
  int seen = 0;
  for (int t0 = lo; t0 < hi; t0 += kBatch) {
    float z[kTok][NE];
    bool on[kTok];
    now.look(t0 + wave, kSumWaves, hi, lane, E, z, on);
    int e_now[kIdx], of_now[kIdx];
#pragma unroll
    for (int q = 0; q < kIdx; ++q) {
      e_now[q] = counted[q] ? expert[q] : -1;
      of_now[q] = of[q];
    }
    if (t0 + kBatch < hi) load(t0 + kBatch);
    Scores<NE, SOFTMAX> sc[kTok];
    score_tokens<NE, SOFTMAX>(z, lane, E, sc);
    float inv[kTok];
#pragma unroll
    for (int t = 0; t < kTok; ++t) inv[t] = on[t] && sc[t].total != 0.0f ? 1.0f / sc[t].total : 0.0f;
    const int stop = min(t0 + kBatch, hi);
    for (; s < a.n_seqs; ++s) {
      int begin, end;
      bounds.of(a, s, begin, end);
      if (!ALONE && begin >= stop) break;
      if (begin >= end) {
        if (ALONE) finish_sequence(a, s, threadIdx.x, (int)threadIdx.x < E, 0, 0.0, 0.0, 0.0, loss, counts, coef);
        continue;
      }
#pragma unroll
      for (int t = 0; t < kTok; ++t) {
        const int tok = t0 + wave + t * kSumWaves;
        if (tok < begin || tok >= end) continue;  // (a factor of 0 would let a NaN of another sequence through)
#pragma unroll
        for (int i = 0; i < NE; ++i) acc[i] = __builtin_fmaf(sc[t].v[i], inv[t], acc[i]);
        seen += on[t] ? 1 : 0;
      }
#pragma unroll
      for (int q = 0; q < kIdx; ++q)
        if ((uint32_t)e_now[q] < (uint32_t)E && of_now[q] >= begin && of_now[q] < end) atomicAdd(&hist[e_now[q]], 1);
      if (!ALONE && end > stop && stop < hi) break;  // goes on in the workgroup's next batch
      // the piece ends: its sums to its slot
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        mass[wave][lane + 64 * i] = acc[i];
        acc[i] = 0.0f;
      }
      if (lane == 0) atomicAdd(&valid, seen);
      seen = 0;
      __syncthreads();
      static_assert(64 * NE <= kSumThreads, "an expert a thread");
      const int e = threadIdx.x;
      float m = 0.0f;
      int c = 0;
      const int valid_now = valid;
      if (e < E) {
#pragma unroll
        for (int w = 0; w < kSumWaves; ++w) m += mass[w][e];
        c = hist[e];
        hist[e] = 0;
      }
      if constexpr (ALONE) {
        double sums[2] = {(double)c, (double)c * (double)m};
        block_totals(sums, totals);
        finish_sequence(a, s, e, e < E, c, (double)valid_now, sums[0], sums[1], loss, counts, coef);
      } else {
        float *slot = slots + (size_t)(blockIdx.x + s) * slot_words(E);
        int *cnt = reinterpret_cast<int *>(slot + E);
        if (e < E) {
          slot[e] = m;
          cnt[e] = c;
        }
        if (e == 0) cnt[E] = valid_now;
      }
      __syncthreads();
      if (threadIdx.x == 0) valid = 0;
      __syncthreads();
      if (!ALONE && end > stop) break;  // the workgroup's last batch
    }
  }
}

// One workgroup per sequence: its pieces' sums, then loss, counts and coef.
// The 1024 threads are 1024 / 64NE groups over the pieces, a column each.
template <int NE>
__global__ __launch_bounds__(1024) void balance_finish_kernel(coli_moe_balance_t a, int chunk_tokens,
                                                              const float *slots, float *loss, int32_t *counts,
                                                              float *coef) {
  constexpr int kCols = 64 * NE, kGroups = 1024 / kCols, kAhead = 8;
  __shared__ double mass[1024];
  __shared__ int cnts[1024];
  __shared__ double totals[3][16];
  const int s = blockIdx.x, E = a.n_experts, col = threadIdx.x % kCols, grp = threadIdx.x / kCols;
  const int begin = seq_at(a, s), end = seq_at(a, s + 1);
  const size_t words = slot_words(E);
  double m = 0.0;
  int c = 0, v = 0;
  if (begin < end) {
    const int first = begin / chunk_tokens, last = (end - 1) / chunk_tokens;
    for (int p0 = first + grp; p0 <= last; p0 += kGroups * kAhead) {
      float part[kAhead];
      int cnt[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {  // kAhead pieces' loads in flight
        const int p = p0 + q * kGroups;
        const float *slot = slots + (size_t)(min(p, last) + s) * words;
        part[q] = slot[min(col, E - 1)];
        cnt[q] = reinterpret_cast<const int *>(slot)[E + min(col, E - 1)];
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        if (p0 + q * kGroups <= last && col < E) {
          m += (double)part[q];
          c += cnt[q];
        }
    }
    for (int p = first + (int)threadIdx.x; p <= last; p += 1024)
      v += reinterpret_cast<const int *>(slots + (size_t)(p + s) * words)[2 * E];
  }
  mass[threadIdx.x] = m;
  cnts[threadIdx.x] = c;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
      m += mass[g * kCols + col];
      c += cnts[g * kCols + col];
    }
  } else {
    m = 0.0;
    c = 0;
  }
  // valid tokens, kept assignments (whole numbers, exact) and their product with the shares
  double sums[3] = {(double)v, (double)c, (double)c * m};
  block_totals(sums, totals);
  finish_sequence(a, s, col, grp == 0 && col < E, c, sums[0], sums[1], sums[2], loss, counts, coef);
}

template <int NE, bool SOFTMAX>
__global__ __launch_bounds__(64 * kGradWaves) void balance_grad_kernel(coli_moe_balance_t a, const float *coef,
                                                                       const float *dloss, float *dlogits,
                                                                       int64_t stride) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), E = a.n_experts;
  const int lo = (blockIdx.x * kGradWaves + wave) * kTok, hi = min(lo + kTok, a.tokens);  // the wave's tokens
  if (lo >= hi) return;
  Bounds bounds;
  bounds.load(a, 0);
  Tokens<NE> tokens;
  tokens.load(a, lo, 1, hi, lane);
  int s = bounds.seek(a, lo);
  float z[kTok][NE];
  bool on[kTok];
  tokens.look(lo, 1, hi, lane, E, z, on);
  Scores<NE, SOFTMAX> sc[kTok];
  score_tokens<NE, SOFTMAX>(z, lane, E, sc);
  for (; s < a.n_seqs; ++s) {
    int begin, end;
    bounds.of(a, s, begin, end);
    if (begin >= hi) break;
    if (begin >= end) continue;
    float c[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) c[i] = lane + 64 * i < E ? coef[(size_t)s * E + lane + 64 * i] : 0.0f;
    const float up = dloss ? dloss[s] : 1.0f;
    float dot[kTok];
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      dot[t] = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) dot[t] = __builtin_fmaf(c[i], sc[t].v[i], dot[t]);
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t) dot[t] = wave_sum(dot[t]);
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      const int tok = lo + t;
      if (tok < begin || tok >= min(end, hi)) continue;
      const bool some = on[t] && sc[t].total != 0.0f;
      const float inv = some ? 1.0f / sc[t].total : 0.0f;
      const float mean = dot[t] * inv;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        if (e < E) dlogits[(int64_t)tok * stride + e] = some ? sc[t].slope[i] * inv * (up * (c[i] - mean)) : 0.0f;
      }
    }
  }
}

// Tokens of one workgroup of the sums: at most kMaxChunks workgroups (their
// pieces are added by one workgroup a sequence), unless that makes a float32
// sum too long.
int chunk_tokens_of(int tokens) {
  constexpr int kMaxChunkTokens = 4096;  // 256 additions a wave
  const int c = std::min((tokens + kMaxChunks - 1) / kMaxChunks, kMaxChunkTokens);
  return (c < 1 ? 1 : (c + kBatchTokens - 1) / kBatchTokens) * kBatchTokens;
}

int chunks_of(int tokens) {
  const int c = chunk_tokens_of(tokens);
  return (tokens + c - 1) / c;
}

// NE: experts a lane holds (1, 2, 4 or 8), as a compile-time constant.
template <class F>
hipError_t by_experts(int E, F &&f) {
  if (E <= 64) return f(std::integral_constant<int, 1>());
  if (E <= 128) return f(std::integral_constant<int, 2>());
  if (E <= 256) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 8>());
}

}  // namespace

size_t balance_workspace_bytes(int tokens, int E, int n_seqs) {
  const size_t slots = (size_t)chunks_of(tokens) + (size_t)n_seqs;
  return slots * slot_words(E) * 4;
}

hipError_t launch_balance(const coli_moe_balance_t &a, float *loss, int32_t *counts, float *coef, float *slots,
                          hipStream_t s) {
  const int chunk = chunk_tokens_of(a.tokens), n = chunks_of(a.tokens);
  return by_experts(a.n_experts, [&](auto ne) {
    constexpr int NE = decltype(ne)::value;
    const auto sums = [&](auto softmax, auto alone) {
      return launch(balance_sums_kernel<NE, decltype(softmax)::value, decltype(alone)::value>, dim3(n),
                    dim3(kSumThreads), 0, s, a, chunk, slots, loss, counts, coef);
    };
    const bool softmax = a.scores == COLI_MOE_SCORES_SOFTMAX;
    if (n == 1 && a.tokens <= kBatchTokens && a.n_seqs <= kAloneSeqs)
      return softmax ? sums(std::true_type(), std::true_type()) : sums(std::false_type(), std::true_type());
    if (n > 0) {
      const hipError_t e =
          softmax ? sums(std::true_type(), std::false_type()) : sums(std::false_type(), std::false_type());
      if (e != hipSuccess) return e;
    }
    return launch(balance_finish_kernel<NE>, dim3(a.n_seqs), dim3(1024), 0, s, a, chunk, slots, loss, counts, coef);
  });
}

hipError_t launch_balance_grad(const coli_moe_balance_t &a, const float *coef, const float *dloss, float *dlogits,
                               int64_t stride, hipStream_t s) {
  const dim3 grid((a.tokens + kTok * kGradWaves - 1) / (kTok * kGradWaves)), block(64 * kGradWaves);
  return by_experts(a.n_experts, [&](auto ne) {
    constexpr int NE = decltype(ne)::value;
    return a.scores == COLI_MOE_SCORES_SOFTMAX
               ? launch(balance_grad_kernel<NE, true>, grid, block, 0, s, a, coef, dloss, dlogits, stride)
               : launch(balance_grad_kernel<NE, false>, grid, block, 0, s, a, coef, dloss, dlogits, stride);
  });
}

}  // namespace coli
