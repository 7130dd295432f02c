// thin.h -- the grouped products for a few rows in all.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

// Rows (N * cap) up to which a product goes this way.  us here against the
// 128-row tiles: one row by 7168 x 2048 6.2 : 9.5, sixteen 8.1 : 9.5, 32 15 : 9.5;
// gate/up of 2048 by 7168 at one row 10.6 : 20.5, sixteen 17.5 : 20.5, of 768 by 2048
// 8.2 : 11.7, 10.3 : 11.7 (eight), 13.0 : 11.7 (sixteen); eight experts with one row
// each 28.6 : 32.7 and (7168 x 2048) 16 : 17, with four each 52 : 43 and 26 : 27.
constexpr int kThinRows = 16;

// y (bf16) or, where h_q is given, the coded activation of the pair of weight
// halves; arguments as moe_expert_gemm's, already checked.
cudaError_t launch_thin_product(int N, int E, int cap, int n, int k, const uint8_t *a_q,
                                const float *a_s, const int32_t *grp_off, const uint8_t *w_q,
                                const float *w_s, uint16_t *y, uint8_t *h_q, float *h_s,
                                int32_t *status, cudaStream_t st);

}  // namespace moe
