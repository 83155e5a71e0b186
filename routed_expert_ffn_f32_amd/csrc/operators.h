// Launchers of the operators around the layer (arguments checked by
// operators.hip; meanings as in coli_moe.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "coli_moe.h"

namespace coli {

hipError_t launch_rmsnorm(const coli_moe_rmsnorm_t &a, hipStream_t s);  // rows >= 1

size_t balance_workspace_bytes(int tokens, int E, int n_seqs);
hipError_t launch_balance(const coli_moe_balance_t &a, float *loss, int32_t *counts, float *coef, float *slots,
                          hipStream_t s);
hipError_t launch_balance_grad(const coli_moe_balance_t &a, const float *coef, const float *dloss, float *dlogits,
                               int64_t stride, hipStream_t s);  // tokens >= 1

hipError_t launch_linear(const coli_moe_linear_t &a, hipStream_t s);  // m, n >= 1
constexpr int kLinearRowsMax = 32;  // rows of x up to which every product takes launch_linear_rows
hipError_t launch_linear_rows(const coli_moe_linear_t &a, hipStream_t s);

}  // namespace coli
