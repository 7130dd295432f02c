// linear.h -- the products of 16-bit rows and weights: their arguments, and which
// kernel takes them, in how many CTAs.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

struct Linear {
    int rows, n, k;  // n: outputs (of each half, where there are two)
    int act;
    const uint16_t *x, *w, *bias, *res;
    uint16_t *y;
    float *yf;
    int32_t *status;
};

// How a product runs.
struct LinearPlan {
    int at;     // rows of a CTA
    int parts;  // CTAs of a cluster that share its k
};

constexpr int kLinearBlock = 64;  // elements of k that a stage holds: 128 bytes

inline LinearPlan linear_plan(int64_t rows, int64_t n, int64_t k, bool pair, bool f32, int sms) {
    const int most = f32 ? 64 : pair ? 128 : 256;
    LinearPlan p = {16, 1};
    while (p.at < most && p.at < rows) p.at *= 2;
    const int64_t tiles = (n + 127) / 128 * ((rows + p.at - 1) / p.at);
    const int64_t blocks = (k + kLinearBlock - 1) / kLinearBlock;
    const int64_t room = (p.at <= 64 ? 2 : 1) * (int64_t)sms;
    while (p.parts < 8 && blocks >= 4 * p.parts && tiles * p.parts * 2 <= room) p.parts *= 2;
    return p;
}

// pair: gate and up halves of w.
cudaError_t launch_linear(const Linear &p, bool pair, cudaStream_t st);

}  // namespace moe
