// C ABI of the operators around the layer: argument checks, then the launch.
#include "operators.h"

#include "coli_moe.h"
#include "element_types.h"
#include "internal.h"
#include "kv_cache.h"

namespace {

bool aligned_to(const void *p, size_t a) { return p && ((uintptr_t)p % a) == 0; }

// A [rows] array of rows of `cols` elements: pointer and stride usable.
// Rows that are written must not overlap (a stride of 0 reads one row for all).
bool rows_ok(const void *p, int type, int64_t stride, int64_t cols, int64_t rows, bool written) {
  constexpr int64_t kMaxOffset = (int64_t)1 << 56;  // elements; no array is that long
  return aligned_to(p, coli::type_bytes(type)) &&
         (rows <= 1 || (stride >= 0 && stride <= kMaxOffset / rows && (!written || stride >= cols)));
}

struct Rows {
  const void *p;
  int64_t ld, rows;
};

}  // namespace

extern "C" {

int coli_moe_rmsnorm(const coli_moe_rmsnorm_t *a, void *stream) {
  using namespace coli;
  if (!a || a->rows < 0 || a->hidden < 1 || a->hidden > 32768) return COLI_MOE_EARG;
  if (!(a->eps >= 0.0f && a->eps <= 0x1.fffffep+127f)) return COLI_MOE_EARG;
  if (!float_type(a->x_type) || (!float_type(a->out_type) && !byte_type(a->out_type))) return COLI_MOE_EARG;
  if (byte_type(a->out_type) ? a->group != 0 && a->group != 64 && a->group != 128 : a->group != 0)
    return COLI_MOE_EARG;
  if ((a->residual == nullptr) != (a->residual_out == nullptr)) return COLI_MOE_EARG;
  if (a->residual && !float_type(a->residual_type)) return COLI_MOE_EARG;
  if (a->weight && !float_type(a->weight_type)) return COLI_MOE_EARG;
  if (a->rows == 0) return COLI_MOE_OK;
  if (!rows_ok(a->x, a->x_type, a->x_stride, a->hidden, a->rows, false) ||
      !rows_ok(a->out, a->out_type, a->out_stride, a->hidden, a->rows, true))
    return COLI_MOE_EARG;
  if (a->residual && (!rows_ok(a->residual, a->residual_type, a->residual_stride, a->hidden, a->rows, false) ||
                      !rows_ok(a->residual_out, a->residual_type, a->residual_out_stride, a->hidden, a->rows, true)))
    return COLI_MOE_EARG;
  // in place is element for element, or the rows would overwrite each other's input
  if (a->residual && a->residual == a->residual_out && a->rows > 1 && a->residual_stride != a->residual_out_stride)
    return COLI_MOE_EARG;
  if (a->out == a->x && (a->out_type != a->x_type || (a->rows > 1 && a->out_stride != a->x_stride)))
    return COLI_MOE_EARG;
  if (a->residual_out && (a->residual_out == a->out || a->residual == a->out ||
                          (a->residual_out == a->x && (a->residual_type != a->x_type ||
                                                       (a->rows > 1 && a->residual_out_stride != a->x_stride)))))
    return COLI_MOE_EARG;
  if (a->weight && !aligned_to(a->weight, type_bytes(a->weight_type))) return COLI_MOE_EARG;
  if (byte_type(a->out_type)) {
    const int64_t n = a->group ? (a->hidden + a->group - 1) / a->group : 1;
    if (!rows_ok(a->scales, COLI_MOE_F32, a->scales_stride, n, a->rows, true)) return COLI_MOE_EARG;
  }
  return launch_rmsnorm(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? COLI_MOE_OK : COLI_MOE_EDEVICE;
}

int coli_moe_linear(const coli_moe_linear_t *a, void *stream) {
  using namespace coli;
  constexpr int32_t kMaxRows = 1 << 22, kMaxK = 1 << 16;
  constexpr int64_t kMaxRowBytes = (int64_t)1 << 23;  // a tile's row offsets are 32-bit
  if (!a || a->m < 0 || a->m > kMaxRows || a->n < 1 || a->n > kMaxRows || a->k < 1 || a->k > kMaxK)
    return COLI_MOE_EARG;
  const bool bytes = byte_type(a->type);
  if (!bytes && a->type != COLI_MOE_BF16 && a->type != COLI_MOE_F16) return COLI_MOE_EARG;
  if (!float_type(a->out_type) || a->act < COLI_MOE_ACT_NONE || a->act > COLI_MOE_ACT_SWIGLU) return COLI_MOE_EARG;
  if (a->bias && !float_type(a->bias_type)) return COLI_MOE_EARG;
  const int64_t esz = (int64_t)type_bytes(a->type);
  if (a->k * esz % 16) return COLI_MOE_EARG;
  if (a->m == 0) return COLI_MOE_OK;
  const int64_t wrows = a->act == COLI_MOE_ACT_SWIGLU ? 2 * (int64_t)a->n : a->n;
  for (const auto &[p, ld, rows] : {Rows{a->x, a->ldx, a->m}, Rows{a->w, a->ldw, wrows}})
    if (!aligned_to(p, 16) ||
        (rows > 1 && (ld < 0 || ld > kMaxRowBytes || ld * esz > kMaxRowBytes || ld * esz % 16)))
      return COLI_MOE_EARG;
  if (bytes ? !aligned_to(a->x_scale, 4) || !aligned_to(a->w_scale, 4) : a->x_scale || a->w_scale)
    return COLI_MOE_EARG;
  if (a->bias && !aligned_to(a->bias, type_bytes(a->bias_type))) return COLI_MOE_EARG;
  if (!rows_ok(a->out, a->out_type, a->ldo, a->n, a->m, true)) return COLI_MOE_EARG;
  if (a->residual && !rows_ok(a->residual, a->out_type, a->ldr, a->n, a->m, false)) return COLI_MOE_EARG;
  if (a->residual == a->out && a->m > 1 && a->ldr != a->ldo) return COLI_MOE_EARG;
  if (a->out == a->x || a->out == a->w) return COLI_MOE_EARG;
  return launch_linear(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? COLI_MOE_OK : COLI_MOE_EDEVICE;
}

}  // extern "C"

namespace {

constexpr int32_t kMaxSeqs = 65536, kMaxTokens = 1 << 26;

int balance_check(const coli_moe_balance_t *a) {
  if (!a || a->tokens < 0 || a->tokens > kMaxTokens || a->n_seqs < 1 || a->n_seqs > kMaxSeqs) return COLI_MOE_EARG;
  if (a->n_experts < 1 || a->n_experts > coli::kMaxExperts || a->top_k < 1 || a->top_k > a->n_experts ||
      a->top_k > coli::kMaxTopK)
    return COLI_MOE_EROUTING;
  if (a->scores != COLI_MOE_SCORES_SIGMOID && a->scores != COLI_MOE_SCORES_SOFTMAX) return COLI_MOE_EARG;
  if (a->seq_offsets ? !aligned_to(a->seq_offsets, 4) : a->n_seqs != 1) return COLI_MOE_EARG;
  if (a->tokens > 0 && !rows_ok(a->logits, COLI_MOE_F32, a->logits_stride, a->n_experts, a->tokens, false))
    return COLI_MOE_EARG;
  return COLI_MOE_OK;
}

}  // namespace

extern "C" {

size_t coli_moe_balance_workspace_bytes(int32_t tokens, int32_t n_experts, int32_t n_seqs) {
  if (tokens < 0 || tokens > kMaxTokens || n_experts < 1 || n_experts > coli::kMaxExperts) return 0;
  if (n_seqs < 1 || n_seqs > kMaxSeqs) return 0;
  return coli::balance_workspace_bytes(tokens, n_experts, n_seqs);
}

int coli_moe_balance(const coli_moe_balance_t *a, float *loss, int32_t *counts, float *coef, void *workspace,
                     size_t workspace_bytes, void *stream) {
  const int code = balance_check(a);
  if (code != COLI_MOE_OK) return code;
  if (a->tokens > 0 && !aligned_to(a->idx, 4)) return COLI_MOE_EARG;
  if ((int64_t)a->tokens * a->top_k > INT32_MAX) return COLI_MOE_EARG;  // counts are int32
  if (!aligned_to(loss, 4) || !aligned_to(counts, 4) || !aligned_to(coef, 4) || !aligned_to(workspace, 16))
    return COLI_MOE_EARG;
  if (workspace_bytes < coli::balance_workspace_bytes(a->tokens, a->n_experts, a->n_seqs)) return COLI_MOE_ECAPACITY;
  return coli::launch_balance(*a, loss, counts, coef, static_cast<float *>(workspace),
                              static_cast<hipStream_t>(stream)) == hipSuccess
             ? COLI_MOE_OK
             : COLI_MOE_EDEVICE;
}

int coli_moe_balance_grad(const coli_moe_balance_t *a, const float *coef, const float *dloss, float *dlogits,
                          int64_t dlogits_stride, void *stream) {
  const int code = balance_check(a);
  if (code != COLI_MOE_OK) return code;
  if (!aligned_to(coef, 4) || (dloss && !aligned_to(dloss, 4))) return COLI_MOE_EARG;
  if (a->tokens == 0) return COLI_MOE_OK;
  if (!rows_ok(dlogits, COLI_MOE_F32, dlogits_stride, a->n_experts, a->tokens, true)) return COLI_MOE_EARG;
  return coli::launch_balance_grad(*a, coef, dloss, dlogits, dlogits_stride, static_cast<hipStream_t>(stream)) ==
                 hipSuccess
             ? COLI_MOE_OK
             : COLI_MOE_EDEVICE;
}

}  // extern "C"

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;

// A [tokens][heads] array of heads of `dim` elements: pointer and strides
// usable.  Heads that are written must not overlap.
bool heads_ok(const void *p, int type, int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim,
              bool written) {
  if (!aligned_to(p, coli::type_bytes(type))) return false;
  if ((tokens > 1 && (token < 0 || token > kMaxStride)) || (heads > 1 && (head < 0 || head > kMaxStride))) return false;
  if (!written) return true;
  if ((heads > 1 && head < dim) || (tokens > 1 && token < dim)) return false;
  // one stride steps over the whole of the other
  return tokens <= 1 || heads <= 1 || token >= (heads - 1) * head + dim || head >= (tokens - 1) * token + dim;
}

// Whether [a, a + n) and [b, b + m) bytes have any in common.
bool ranges_meet(const void *a, size_t n, const void *b, size_t m) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y ? y - x < n : x - y < m;
}

// A [tokens][heads] array of heads, heads_ok, and one that is written.
struct Heads {
  const void *p;
  int64_t token, head;
};

// Whether an element of `in` is one of `out`.  Both may be views of one buffer
// whose elements lie between each other's: exact where in's heads are within a
// token as out's are (or its tokens within a head), the steps from token to token
// are equal (or in's 0) and those from head to head too, or the heads at most
// 4096; else any two that reach into each other's range count.
bool heads_meet(Heads in, Heads out, int type, int64_t tokens, int64_t heads, int64_t dim) {
  const int64_t size = (int64_t)coli::type_bytes(type);
  auto bytes = [&](const Heads &a) {  // strides are up to kMaxStride: within 2^68
    const __int128 n = ((tokens > 1 ? (__int128)(tokens - 1) * a.token : 0) +
                        (heads > 1 ? (__int128)(heads - 1) * a.head : 0) + dim) * size;
    return n > INT64_MAX ? (size_t)INT64_MAX : (size_t)n;
  };
  if (!ranges_meet(in.p, bytes(in), out.p, bytes(out))) return false;
  // how many steps each side takes, and how long they are; steps of 0 are none
  struct Level {
    int64_t in, in_step, out, out_step;
  };
  auto level = [](int64_t n, int64_t a, int64_t b) { return Level{n == 1 || a == 0 ? 1 : n, a, n, n == 1 ? 0 : b}; };
  Level outer = level(tokens, in.token, out.token), inner = level(heads, in.head, out.head);
  if (tokens > 1 && (heads == 1 || out.token < out.head)) {
    const Level t = outer;
    outer = inner;
    inner = t;
  }
  if (outer.out > 1 && ((outer.in > 1 && outer.in_step != outer.out_step) ||
                        (__int128)(inner.in - 1) * inner.in_step + dim > outer.out_step))
    return true;
  // the number of steps, of those there are, that brings d to 0 or next below (k 0), or above (1)
  auto near = [](int64_t d, int64_t step, int64_t least, int64_t most, int k) {
    if (step == 0) return (int64_t)0;
    const int64_t q = -d / step - (-d % step < 0 ? 1 : 0) + k;
    return q > most ? most : q < least ? least : q;
  };
  // out - in in elements
  const int64_t delta = ((intptr_t)out.p - (intptr_t)in.p) / size;
  const bool alike = inner.in == 1 || inner.in_step == inner.out_step;
  if (!alike && inner.out > 4096) return true;  // more than is worth a look
  for (int k = 0; k < 2; ++k) {
    const int64_t r = delta + near(delta, outer.out_step, 1 - outer.in, outer.out - 1, k) * outer.out_step;
    for (int n = 0; n < 2; ++n) {
      if (alike) {
        const int64_t d = r + near(r, inner.out_step, 1 - inner.in, inner.out - 1, n) * inner.out_step;
        if (d > -dim && d < dim) return true;
        continue;
      }
      for (int64_t j = 0; j < inner.out; ++j) {
        const int64_t at = r + j * inner.out_step;  // and in's step next to it
        const int64_t d = at + near(at, inner.in_step, 1 - inner.in, 0, n) * inner.in_step;
        if (d > -dim && d < dim) return true;
      }
    }
  }
  return false;
}

int kv_check(const coli_moe_kv_t *kv) {
  if (!kv || kv->n_pages < 1 || kv->kv_heads < 1 || kv->kv_heads > 1024) return COLI_MOE_EARG;
  if (kv->page_size < 16 || kv->page_size > 256 || (kv->page_size & (kv->page_size - 1))) return COLI_MOE_EARG;
  return kv->head_dim == 64 || kv->head_dim == 128 || kv->head_dim == 256 ? COLI_MOE_OK : COLI_MOE_EARG;
}

bool kv_pointers_ok(const coli_moe_kv_t *kv) {
  return aligned_to(kv->k_codes, 16) && aligned_to(kv->k_scales, 16) && aligned_to(kv->v_codes, 16) &&
         aligned_to(kv->v_scales, 16) && (!kv->weights || aligned_to(kv->weights, 16));
}

constexpr int32_t kMaxKvTokens = 1 << 22;

int kv_rows_check(const coli_moe_kv_t *kv, const coli_moe_kv_rows_t *r) {
  if (!r || r->seqs < 1 || r->seqs > kMaxSeqs || r->table_width < 1) return COLI_MOE_EARG;
  return (int64_t)r->table_width * kv->page_size <= (int64_t)1 << 30 ? COLI_MOE_OK : COLI_MOE_EARG;
}

int kv_tokens_check(const coli_moe_kv_rows_t *r) {
  if (r->tokens < 0 || r->tokens > kMaxKvTokens) return COLI_MOE_EARG;
  return r->offsets || r->tokens == r->seqs ? COLI_MOE_OK : COLI_MOE_EARG;
}

bool kv_row_pointers_ok(const coli_moe_kv_rows_t *r) {
  return aligned_to(r->table, 4) && aligned_to(r->lengths, 4) && (!r->offsets || aligned_to(r->offsets, 4)) &&
         (r->seqs == 1 || (r->table_stride >= 0 && r->table_stride <= kMaxStride));
}

// Arguments of append and (written) of read.
int kv_values_check(const coli_moe_kv_t *kv, const coli_moe_kv_rows_t *r, const coli_moe_kv_values_t *a, bool written) {
  int code = kv_check(kv);
  if (code == COLI_MOE_OK) code = kv_rows_check(kv, r);
  if (code == COLI_MOE_OK) code = kv_tokens_check(r);
  if (code != COLI_MOE_OK) return code;
  if (!a || !coli::float_type(a->type) || a->clear < 0 || a->clear > (written ? 1 : 0)) return COLI_MOE_EARG;
  if (!kv_pointers_ok(kv) || !kv_row_pointers_ok(r)) return COLI_MOE_EARG;
  if (r->tokens == 0) return COLI_MOE_OK;
  if (!heads_ok(a->k, a->type, r->tokens, a->k_token, kv->kv_heads, a->k_head, kv->head_dim, written) ||
      !heads_ok(a->v, a->type, r->tokens, a->v_token, kv->kv_heads, a->v_head, kv->head_dim, written))
    return COLI_MOE_EARG;
  return written && heads_meet({a->k, a->k_token, a->k_head}, {a->v, a->v_token, a->v_head}, a->type, r->tokens,
                               kv->kv_heads, kv->head_dim)
             ? COLI_MOE_EARG
             : COLI_MOE_OK;
}

bool finite(float v) { return v >= -0x1.fffffep+127f && v <= 0x1.fffffep+127f; }

int kv_attention_check(const coli_moe_kv_t *kv, const coli_moe_kv_rows_t *r, const coli_moe_kv_attention_t *a) {
  int code = kv_check(kv);
  if (code == COLI_MOE_OK) code = kv_rows_check(kv, r);
  if (code == COLI_MOE_OK) code = kv_tokens_check(r);
  if (code != COLI_MOE_OK) return code;
  if (!a || (a->type != COLI_MOE_BF16 && a->type != COLI_MOE_F16)) return COLI_MOE_EARG;
  if (a->q_heads < kv->kv_heads || a->q_heads % kv->kv_heads || a->q_heads / kv->kv_heads > 256) return COLI_MOE_EARG;
  return a->window >= 0 && (a->clear & ~1) == 0 && finite(a->scale) ? COLI_MOE_OK : COLI_MOE_EARG;
}

int launched(hipError_t e) { return e == hipSuccess ? COLI_MOE_OK : COLI_MOE_EDEVICE; }

}  // namespace

extern "C" {

int coli_moe_rotary(const coli_moe_rotary_t *a, void *stream) {
  using namespace coli;
  if (!a || a->tokens < 0 || a->tokens > kMaxTokens || a->heads < 1 || a->heads > 4096 || a->dim < 1 || a->dim > 4096)
    return COLI_MOE_EARG;
  if (a->part < 0 || a->part > a->dim || a->part % 2 || !float_type(a->type) || !finite(a->scale)) return COLI_MOE_EARG;
  if ((a->interleaved | a->inverse | a->wide) & ~1) return COLI_MOE_EARG;
  if (a->tokens == 0) return COLI_MOE_OK;
  if (!heads_ok(a->x, a->type, a->tokens, a->x_token, a->heads, a->x_head, a->dim, false) ||
      !heads_ok(a->out, a->type, a->tokens, a->out_token, a->heads, a->out_head, a->dim, true))
    return COLI_MOE_EARG;
  if (!aligned_to(a->positions, a->wide ? 8 : 4) || (a->part > 0 && !aligned_to(a->freq, 4))) return COLI_MOE_EARG;
  const bool in_place = a->out == a->x && (a->tokens == 1 || a->out_token == a->x_token) &&
                        (a->heads == 1 || a->out_head == a->x_head);
  if (!in_place && heads_meet({a->x, a->x_token, a->x_head}, {a->out, a->out_token, a->out_head}, a->type, a->tokens,
                              a->heads, a->dim))
    return COLI_MOE_EARG;
  return launched(launch_rotary(*a, static_cast<hipStream_t>(stream)));
}

int coli_moe_kv_append(const coli_moe_kv_t *kv, const coli_moe_kv_rows_t *rows, const coli_moe_kv_values_t *a,
                       void *stream) {
  const int code = kv_values_check(kv, rows, a, false);
  if (code != COLI_MOE_OK || rows->tokens == 0) return code;
  return launched(coli::launch_kv_append(*kv, *rows, *a, static_cast<hipStream_t>(stream)));
}

int coli_moe_kv_read(const coli_moe_kv_t *kv, const coli_moe_kv_rows_t *rows, const coli_moe_kv_values_t *a,
                     void *stream) {
  const int code = kv_values_check(kv, rows, a, true);
  if (code != COLI_MOE_OK || rows->tokens == 0) return code;
  return launched(coli::launch_kv_read(*kv, *rows, *a, static_cast<hipStream_t>(stream)));
}

size_t coli_moe_kv_attention_workspace_bytes(const coli_moe_kv_t *kv, const coli_moe_kv_rows_t *rows,
                                             const coli_moe_kv_attention_t *a) {
  return kv_attention_check(kv, rows, a) == COLI_MOE_OK ? coli::kv_attention_workspace_bytes(*kv, *rows, *a) : 0;
}

int coli_moe_kv_attention(const coli_moe_kv_t *kv, const coli_moe_kv_rows_t *rows, const coli_moe_kv_attention_t *a,
                          void *workspace, size_t workspace_bytes, void *stream) {
  const int code = kv_attention_check(kv, rows, a);
  if (code != COLI_MOE_OK) return code;
  if (!kv_pointers_ok(kv) || !kv_row_pointers_ok(rows)) return COLI_MOE_EARG;
  if (a->weights_out && (!kv->weights || !aligned_to(a->weights_out, 16))) return COLI_MOE_EARG;
  const size_t bytes = (size_t)kv->n_pages * kv->kv_heads * kv->page_size * sizeof(float);  // of the weights
  if (a->weights_out && a->weights_out != kv->weights && ranges_meet(a->weights_out, bytes, kv->weights, bytes))
    return COLI_MOE_EARG;
  if (rows->tokens == 0) return COLI_MOE_OK;
  if (!heads_ok(a->q, a->type, rows->tokens, a->q_token, a->q_heads, a->q_head, kv->head_dim, false) ||
      !heads_ok(a->out, a->type, rows->tokens, a->out_token, a->q_heads, a->out_head, kv->head_dim, true) ||
      heads_meet({a->q, a->q_token, a->q_head}, {a->out, a->out_token, a->out_head}, a->type, rows->tokens, a->q_heads,
                 kv->head_dim) ||
      !aligned_to(workspace, 16))
    return COLI_MOE_EARG;
  if (workspace_bytes < coli::kv_attention_workspace_bytes(*kv, *rows, *a)) return COLI_MOE_ECAPACITY;
  return launched(coli::launch_kv_attention(*kv, *rows, *a, workspace, static_cast<hipStream_t>(stream)));
}

int coli_moe_kv_evict(const coli_moe_kv_t *kv, const coli_moe_kv_rows_t *rows, const coli_moe_kv_evict_t *a,
                      void *stream) {
  int code = kv_check(kv);
  if (code == COLI_MOE_OK) code = kv_rows_check(kv, rows);
  if (code != COLI_MOE_OK) return code;
  if (!a || a->into_width < 1 || (int64_t)a->into_width * kv->page_size > (int64_t)1 << 30) return COLI_MOE_EARG;
  if (a->keep < 1 || a->keep > a->into_width * kv->page_size) return COLI_MOE_EARG;
  if (a->first < 0 || a->recent < 0 || a->first > a->keep || a->recent > a->keep - a->first) return COLI_MOE_EARG;
  if (!kv_pointers_ok(kv) || !kv->weights || !kv_row_pointers_ok(rows)) return COLI_MOE_EARG;
  if (!aligned_to(a->into, 4) || !aligned_to(a->kept, 4) || !aligned_to(a->new_lengths, 4)) return COLI_MOE_EARG;
  if (rows->seqs > 1 && (a->into_stride < 0 || a->into_stride > kMaxStride)) return COLI_MOE_EARG;
  const size_t lengths = (size_t)rows->seqs * 4, kept = lengths * kv->kv_heads * a->keep;
  if (a->into == rows->table || ranges_meet(a->new_lengths, lengths, rows->lengths, lengths) ||
      ranges_meet(a->kept, kept, rows->lengths, lengths) || ranges_meet(a->kept, kept, a->new_lengths, lengths))
    return COLI_MOE_EARG;
  return launched(coli::launch_kv_evict(*kv, *rows, *a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
