// C ABI of the operators around the layer: argument checks, then the launch.
#include "operators.h"

#include "coli_moe.h"
#include "element_types.h"
#include "internal.h"

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
