// linear.h -- the products of 16-bit rows and weights: their arguments and launchers.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "linear_plan.h"

namespace moe {

struct Linear {
    int rows, n, k;  // n: outputs (of each half, where there are two)
    int act;
    const uint16_t *x, *w, *bias, *res;
    uint16_t *y;
    float *yf;
    int32_t *status;
};

// pair: gate and up halves of w.
cudaError_t launch_linear_tiles(const Linear &p, bool pair, const LinearPlan &plan, cudaStream_t st);
cudaError_t launch_linear_ragged(const Linear &p, bool pair, const LinearPlan &plan,
                                 cudaStream_t st);
cudaError_t launch_linear(const Linear &p, bool pair, cudaStream_t st);

}  // namespace moe
