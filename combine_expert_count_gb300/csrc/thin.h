// thin.h -- the grouped products for few rows.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "launch.h"

namespace moe {

// Rows of an expert that meet its weights at a time, a product's columns.  More are
// several CTAs, whose reads of the weights meet in L2.
constexpr int kThinRowsAt = 16;

// Whether a product goes this way: few rows in all, or few enough groups of 16 of
// an expert that all their CTAs are on the SMs at once.  us here against the
// 128-row tiles: 7168 x 2048 one row 7.3 : 9.4, 32 rows 8.5 : 9.8, 96 (not so) 16.4 :
// 10.1; 7168 x 7168 32 rows 16.1 : 19.2, 48 (not so) 22.9 : 19.3; 16 experts with
// 32 rows in all 39 : 41; 512 x 2048 256 rows 6.2 : 8.7; 128 x 7168 1024 rows 10.4 :
// 17.4; gate/up of 2048 by 7168 16 rows 11.7 : 20.3, 64 rows 14.1 : 20.3.
inline bool few_rows(int64_t N, int64_t cap, int64_t E, int64_t n) {
    const int64_t rows = N * cap;
    const int64_t units = (rows < E ? rows : E) * ((cap + kThinRowsAt - 1) / kThinRowsAt);
    return rows <= 2 * kThinRowsAt || (n >> 7) * units < sm_count();
}

// y (bf16) or, where h_q is given, the coded activation of the pair of weight
// halves; arguments as moe_expert_gemm's, already checked.
cudaError_t launch_thin_product(int N, int E, int cap, int n, int k, const uint8_t *a_q,
                                const float *a_s, const int32_t *grp_off, const uint8_t *w_q,
                                const float *w_s, uint16_t *y, uint8_t *h_q, float *h_s,
                                int32_t *status, cudaStream_t st);

}  // namespace moe
