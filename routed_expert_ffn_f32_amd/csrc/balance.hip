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
// give the loads and the reductions something to overlap with.
//
// Sums over tokens: a workgroup owns a run of consecutive tokens (a chunk)
// and visits the pieces of sequences in it.  A piece's sums go to slot
// (chunk + sequence) of the workspace: going through the tokens in order,
// each next piece has a larger chunk, a larger sequence, or both, so no two
// pieces share a slot.  A second launch adds a sequence's pieces in float64
// in a fixed order.  No atomics on floats: the same call gives the same bits.
#include "internal.h"
#include "wave.h"

#include <type_traits>

#include "coli_moe.h"
#include "operators.h"
#include "scalar_math.h"

namespace coli {
namespace {

constexpr int kTok = 4;              // tokens a wave works on at once
constexpr int kSumWaves = 8;         // waves of a workgroup of the sums
constexpr int kSumThreads = 64 * kSumWaves;
constexpr int kMaxChunks = 512;      // workgroups of the sums
constexpr int kMinChunkTokens = 32;  // one batch of four tokens a wave
constexpr int kGradTokens = 32;      // tokens of a workgroup of the gradient
constexpr int kGradWaves = 4;

// Largest over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

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
    for (int t = 0; t < kTok; ++t) top[t] = wave_max(top[t]);
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      float v, d;
      if constexpr (SOFTMAX) {
        // all -Inf: nothing to subtract, every share 0
        v = z[t][i] == -__builtin_inff() ? 0.0f : exp_neg(z[t][i] - top[t]);
        d = v;
      } else {
        // a = exp(-|z|): sigma and sigma (1 - sigma) = a / (1 + a)^2 without
        // overflow or cancellation
        const float a = exp_neg(-fabsf(z[t][i]));
        const float q = 1.0f / (1.0f + a);
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

// First sequence that ends behind token t (n_seqs: none).
__device__ __forceinline__ int first_seq(const coli_moe_balance_t &a, int t) {
  int lo = 0, hi = a.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq_at(a, mid + 1) > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

template <int NE>
__device__ __forceinline__ void load_tokens(const coli_moe_balance_t &a, int t0, int step, int end, int lane,
                                            float (&z)[kTok][NE], bool (&on)[kTok]) {
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    const int tok = t0 + t * step;
    on[t] = tok < end && (!a.mask || a.mask[tok]);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      z[t][i] = on[t] && e < a.n_experts ? a.logits[(int64_t)tok * a.logits_stride + e] : -__builtin_inff();
    }
  }
}

// Sums of one piece: share sums [E], counts [E], valid tokens (as float32
// words: E floats, then E + 1 ints).
__host__ __device__ inline size_t slot_words(int E) { return 2 * (size_t)E + 1; }

template <int NE, bool SOFTMAX>
__global__ __launch_bounds__(kSumThreads) void balance_sums_kernel(coli_moe_balance_t a, int chunk_tokens,
                                                                   float *slots) {
  __shared__ float mass[kSumWaves][64 * NE];
  __shared__ int hist[64 * NE];
  __shared__ int valid;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), E = a.n_experts, k = a.top_k;
  const int lo = blockIdx.x * chunk_tokens, hi = min(lo + chunk_tokens, a.tokens);
  for (int s = first_seq(a, lo); s < a.n_seqs; ++s) {
    const int begin = max(seq_at(a, s), lo), end = min(seq_at(a, s + 1), hi);
    if (begin >= hi) break;
    if (begin >= end) continue;
    for (int i = threadIdx.x; i < E; i += kSumThreads) hist[i] = 0;
    if (threadIdx.x == 0) valid = 0;
    __syncthreads();
    // counts of the kept assignments
    const int n = (end - begin) * k;
    const int32_t *idx = a.idx + (int64_t)begin * k;
    for (int i = threadIdx.x; i < n; i += kSumThreads) {
      const int e = idx[i];
      if ((uint32_t)e < (uint32_t)E && (!a.mask || a.mask[begin + (uint32_t)i / (uint32_t)k])) atomicAdd(&hist[e], 1);
    }
    // shares
    float acc[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) acc[i] = 0.0f;
    int seen = 0;
    for (int t0 = begin + wave; t0 < end; t0 += kTok * kSumWaves) {
      float z[kTok][NE];
      bool on[kTok];
      load_tokens<NE>(a, t0, kSumWaves, end, lane, z, on);
      Scores<NE, SOFTMAX> sc[kTok];
      score_tokens<NE, SOFTMAX>(z, lane, E, sc);
#pragma unroll
      for (int t = 0; t < kTok; ++t) {
        const float inv = on[t] && sc[t].total > 0.0f ? 1.0f / sc[t].total : 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) acc[i] = __builtin_fmaf(sc[t].v[i], inv, acc[i]);
        seen += on[t] ? 1 : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) mass[wave][lane + 64 * i] = acc[i];
    if (lane == 0) atomicAdd(&valid, seen);
    __syncthreads();
    float *slot = slots + (size_t)(blockIdx.x + s) * slot_words(E);
    int *cnt = reinterpret_cast<int *>(slot + E);
    for (int e = threadIdx.x; e < E; e += kSumThreads) {
      float m = 0.0f;
#pragma unroll
      for (int w = 0; w < kSumWaves; ++w) m += mass[w][e];
      slot[e] = m;
      cnt[e] = hist[e];
    }
    if (threadIdx.x == 0) cnt[E] = valid;
    __syncthreads();
  }
}

// Sum of v over a workgroup of 1024 threads, in every thread.
__device__ __forceinline__ double block_sum(double v, double *scratch) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
  for (int i = 0; i < 16; ++i) t += scratch[i];
  return t;
}

// One workgroup per sequence: its pieces' sums, then loss, counts and coef.
// The 1024 threads are 1024 / 64NE groups over the pieces, a column each.
template <int NE>
__global__ __launch_bounds__(1024) void balance_finish_kernel(coli_moe_balance_t a, int chunk_tokens,
                                                              const float *slots, float *loss, int32_t *counts,
                                                              float *coef) {
  constexpr int kCols = 64 * NE, kGroups = 1024 / kCols;
  __shared__ double mass[1024];
  __shared__ int cnts[1024];
  __shared__ double scratch[16];
  const int s = blockIdx.x, E = a.n_experts, col = threadIdx.x % kCols, grp = threadIdx.x / kCols;
  const int begin = seq_at(a, s), end = seq_at(a, s + 1);
  const size_t words = slot_words(E);
  double m = 0.0;
  int c = 0, v = 0;
  if (begin < end) {
    const int first = begin / chunk_tokens, last = (end - 1) / chunk_tokens;
#pragma unroll 4
    for (int p = first + grp; p <= last; p += kGroups) {
      const float *slot = slots + (size_t)(p + s) * words;
      const int *cnt = reinterpret_cast<const int *>(slot + E);
      if (col < E) {
        m += (double)slot[col];
        c += cnt[col];
      }
    }
    for (int p = first + (int)threadIdx.x; p <= last; p += 1024)
      v += reinterpret_cast<const int *>(slots + (size_t)(p + s) * words + E)[E];
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
  const double V = block_sum((double)v, scratch);
  const double N = block_sum((double)c, scratch);
  const double dot = block_sum((double)c * m, scratch);
  const bool some = V > 0.0 && N > 0.0;
  if (threadIdx.x == 0) loss[s] = some ? (float)((double)a.alpha * E * dot / (N * V)) : 0.0f;
  if (grp == 0 && col < E) {
    counts[(size_t)s * E + col] = c;
    coef[(size_t)s * E + col] = some ? (float)((double)a.alpha / V * ((double)c * E / N - 1.0)) : 0.0f;
  }
}

template <int NE, bool SOFTMAX>
__global__ __launch_bounds__(64 * kGradWaves) void balance_grad_kernel(coli_moe_balance_t a, const float *coef,
                                                                       const float *dloss, float *dlogits,
                                                                       int64_t stride) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), E = a.n_experts;
  const int lo = blockIdx.x * kGradTokens, hi = min(lo + kGradTokens, a.tokens);
  for (int s = first_seq(a, lo); s < a.n_seqs; ++s) {
    const int begin = max(seq_at(a, s), lo), end = min(seq_at(a, s + 1), hi);
    if (begin >= hi) break;
    if (begin >= end) continue;
    float c[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      c[i] = e < E ? coef[(size_t)s * E + e] : 0.0f;
    }
    const float up = dloss ? dloss[s] : 1.0f;
    for (int t0 = begin + wave; t0 < end; t0 += kTok * kGradWaves) {
      float z[kTok][NE];
      bool on[kTok];
      load_tokens<NE>(a, t0, kGradWaves, end, lane, z, on);
      Scores<NE, SOFTMAX> sc[kTok];
      score_tokens<NE, SOFTMAX>(z, lane, E, sc);
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
        const int tok = t0 + t * kGradWaves;
        if (tok >= end) continue;
        const bool some = on[t] && sc[t].total > 0.0f;
        const float inv = some ? 1.0f / sc[t].total : 0.0f;
        const float mean = dot[t] * inv, scale = up * inv;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          const int e = lane + 64 * i;
          if (e < E) dlogits[(int64_t)tok * stride + e] = some ? scale * sc[t].slope[i] * (c[i] - mean) : 0.0f;
        }
      }
    }
  }
}

// Tokens of one workgroup of the sums.
int chunk_tokens_of(int tokens) {
  const int c = (tokens + kMaxChunks - 1) / kMaxChunks;
  return c < kMinChunkTokens ? kMinChunkTokens : c;
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
    if (n > 0) {
      const hipError_t e = a.scores == COLI_MOE_SCORES_SOFTMAX
                               ? launch(balance_sums_kernel<NE, true>, dim3(n), dim3(kSumThreads), 0, s, a, chunk, slots)
                               : launch(balance_sums_kernel<NE, false>, dim3(n), dim3(kSumThreads), 0, s, a, chunk, slots);
      if (e != hipSuccess) return e;
    }
    return launch(balance_finish_kernel<NE>, dim3(a.n_seqs), dim3(1024), 0, s, a, chunk, slots, loss, counts, coef);
  });
}

hipError_t launch_balance_grad(const coli_moe_balance_t &a, const float *coef, const float *dloss, float *dlogits,
                               int64_t stride, hipStream_t s) {
  const dim3 grid((a.tokens + kGradTokens - 1) / kGradTokens), block(64 * kGradWaves);
  return by_experts(a.n_experts, [&](auto ne) {
    constexpr int NE = decltype(ne)::value;
    return a.scores == COLI_MOE_SCORES_SOFTMAX
               ? launch(balance_grad_kernel<NE, true>, grid, block, 0, s, a, coef, dloss, dlogits, stride)
               : launch(balance_grad_kernel<NE, false>, grid, block, 0, s, a, coef, dloss, dlogits, stride);
  });
}

}  // namespace coli
