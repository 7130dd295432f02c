// linear.h -- the products of 16-bit rows and weights: their arguments, and which
// kernel takes them, in how many CTAs.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#ifdef MOE_LINEAR_TUNE
#include <cstdlib>
#endif

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
    int width;  // > 0: pairs of CTAs, tiles of 256 rows by so many weight rows
    int at;     // rows of a CTA
    int parts;  // CTAs of a cluster that share its k
};

constexpr int kLinearBlock = 64;  // elements of k that a stage holds: 128 bytes

inline LinearPlan linear_plan(int64_t rows, int64_t n, int64_t k, bool pair, bool f32, int sms) {
    const int most = f32 ? 64 : pair ? 128 : 256;
    LinearPlan p = {0, 16, 1};
    if (rows > 256) p.width = f32 ? 128 : 256;
    while (p.at < most && p.at < rows) p.at *= 2;
    const int64_t tiles = (n + 127) / 128 * ((rows + p.at - 1) / p.at);
    const int64_t blocks = (k + kLinearBlock - 1) / kLinearBlock;
    const int64_t room = (p.at <= 64 ? 2 : 1) * (int64_t)sms;
    if (p.width == 0)
        while (p.parts < 8 && blocks >= 4 * p.parts && tiles * p.parts * 2 <= room) p.parts *= 2;
#ifdef MOE_LINEAR_TUNE
    if (getenv("LW")) p.width = atoi(getenv("LW"));
    if (getenv("LAT")) p.at = atoi(getenv("LAT"));
    if (getenv("LP")) p.parts = atoi(getenv("LP"));
    if (f32 && p.width > 128) p.width = 128;
    if (pair && p.width) p.width = (p.width + 63) / 64 * 64;
    if (!p.width && p.at > most) p.at = most;
    while (p.parts > blocks) p.parts /= 2;
#endif
    return p;
}

// pair: gate and up halves of w.
cudaError_t launch_linear_tiles(const Linear &p, bool pair, const LinearPlan &plan, cudaStream_t st);
cudaError_t launch_linear(const Linear &p, bool pair, cudaStream_t st);

}  // namespace moe
