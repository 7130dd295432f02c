// thin.h -- the grouped products for few rows.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "launch.h"

namespace moe {

// Rows of an expert that meet its weights at a time, a product's columns.  More are
// several CTAs, whose reads of the weights meet in L2.
constexpr int kThinRowsAt = 16;

// Groups of 16 rows of an expert that there can be, at least one for each expert
// with rows.
inline int64_t thin_units(int64_t N, int64_t cap, int64_t E) {
    const int64_t rows = N * cap, used = rows < E ? rows : E;
    return (rows - used) / kThinRowsAt + used;
}

// Whether a product goes this way.  us here against the 128-row tiles:
//   32 rows in all: 7168 x 2048 8.5 : 9.8; 7168 x 7168 16.1 : 19.2; 16 experts of
//   7168 x 2048 39 : 41; gate/up of 2048 by 7168 11.8 : 20.2
//   or all CTAs on the SMs at once: 4096 x 4096, 64 rows 10.6 : 14.1; 128 x 7168, 1024
//   rows 10.4 : 17.4; gate/up of 2048 by 7168, 64 rows 13.9 : 20.3; (not so) 7168 x
//   2048, 96 rows 16.3 : 10.1
//   or at most eight rows an expert, and 512 KB of weights to each CTA: 32 experts'
//   gate/up of 2048 by 7168, 128 rows 145 : 157, of 128 uneven ones of 768 by 2048, 1021
//   rows 64.7 : 65.4; 32 of 2048 x 7168, 256 rows 76.5 : 80.1; (not so, 12 rows each)
//   the last, uneven 83.8 : 80.3; (not so, 96 KB) 128 of 2048 x 768, 512 rows 48 : 43
inline bool few_rows(int64_t N, int64_t cap, int64_t E, int64_t n, int64_t k, bool pair) {
    const int64_t rows = N * cap;
    return rows <= 32 || (n >> 7) * thin_units(N, cap, E) < sm_count() ||
           (rows <= 8 * E && (pair ? 2 : 1) * k >= 4096);
}

// y (bf16) or, where h_q is given, the coded activation of the pair of weight
// halves; arguments as moe_expert_gemm's, already checked.
cudaError_t launch_thin_product(int N, int E, int cap, int n, int k, const uint8_t *a_q,
                                const float *a_s, const int32_t *grp_off, const uint8_t *w_q,
                                const float *w_s, uint16_t *y, uint8_t *h_q, float *h_s,
                                int32_t *status, cudaStream_t st);

}  // namespace moe
