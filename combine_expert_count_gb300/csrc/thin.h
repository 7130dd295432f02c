// thin.h -- the grouped products for few rows.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "plan.h"

namespace moe {

// y (bf16) or, where h_q is given, the coded activation of the pair of weight
// halves; arguments as moe_expert_gemm's, already checked.
cudaError_t launch_thin_product(const ProductPlan &plan, int N, int E, int cap, int n, int k,
                                const uint8_t *a_q, const float *a_s, const int32_t *grp_off,
                                const uint8_t *w_q, const float *w_s, uint16_t *y, uint8_t *h_q,
                                float *h_s, int32_t *status, cudaStream_t st);

}  // namespace moe
