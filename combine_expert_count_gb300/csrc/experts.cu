// experts.cu -- the experts' products over the grouped rows: moe_expert_gemm
// and moe_expert_gemm_swiglu.
#include "bf16.cuh"
#include "check.h"
#include "coding.cuh"
#include "launch.h"
#include "mma8.cuh"
#include "trace.h"

namespace moe {

struct Product {
    int N, E, cap, n, k;
    const uint8_t *a_q;
    const float *a_s;
    const int32_t *grp_off;
    const uint8_t *w_q;
    const float *w_s;
    uint16_t *y;
    uint8_t *h_q;
    float *h_s;
};

// First row and row count of expert e within its rank's rows, clipped.
__device__ __forceinline__ int2 group_rows(const Product &p, int e) {
    if (!p.grp_off) return make_int2(0, p.cap);
    const int Er = p.E / p.N, r = e / Er, j = e - r * Er;
    const int32_t *off = p.grp_off + (size_t)r * (Er + 1) + j;
    const int b = min(max(__ldg(off), 0), p.cap), t = min(max(__ldg(off + 1), b), p.cap);
    return make_int2(b, t - b);
}

// One CTA: 16 rows of one expert by 128 outputs (kSwiglu: 128 of the gate and
// the same 128 of the up), warp w taking 16 of each.
template <bool kSwiglu>
__global__ void __launch_bounds__(256) k_product_simple(const Product p) {
    __shared__ uint32_t wmax[8][16];
    const int e = blockIdx.z, Er = p.E / p.N;
    const int2 g = group_rows(p, e);
    const int r0 = blockIdx.x * 16;
    if (r0 >= g.y) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, t4 = lane & 3;
    const size_t row0 = (size_t)(e / Er) * p.cap + g.x + r0;
    const int Kb = p.k >> 7, nb = p.n >> 7;
    constexpr int kHalves = kSwiglu ? 2 : 1;
    float acc[kHalves][2][4] = {};
    for (int b = 0; b < Kb; ++b) {
        uint32_t a[4][4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rr = gid + (i & 1) * 8;
                a[kk][i] = r0 + rr < g.y
                               ? *reinterpret_cast<const uint32_t *>(
                                     p.a_q + (row0 + rr) * p.k + b * 128 + kk * 32 + t4 * 4 + (i >> 1) * 16)
                               : 0u;
            }
        const float s0 = r0 + gid < g.y ? __ldg(p.a_s + (row0 + gid) * Kb + b) : 0.0f;
        const float s1 = r0 + gid + 8 < g.y ? __ldg(p.a_s + (row0 + gid + 8) * Kb + b) : 0.0f;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const int blk = blockIdx.y + h * (nb / 2);
            const float ws = __ldg(p.w_s + ((size_t)e * nb + blk) * Kb + b);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint8_t *w = p.w_q + ((size_t)e * p.n + blk * 128 + warp * 16 + j * 8 + gid) * p.k + b * 128 + t4 * 4;
                float c[4] = {};
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_e4m3(c, a[kk], *reinterpret_cast<const uint32_t *>(w + kk * 32),
                             *reinterpret_cast<const uint32_t *>(w + kk * 32 + 16));
                acc[h][j][0] = __fmaf_rn(s0 * ws, c[0], acc[h][j][0]);
                acc[h][j][1] = __fmaf_rn(s0 * ws, c[1], acc[h][j][1]);
                acc[h][j][2] = __fmaf_rn(s1 * ws, c[2], acc[h][j][2]);
                acc[h][j][3] = __fmaf_rn(s1 * ws, c[3], acc[h][j][3]);
            }
        }
    }
    if constexpr (!kSwiglu) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (r0 + gid + i * 8 < g.y)
                    *reinterpret_cast<uint32_t *>(p.y + (row0 + gid + i * 8) * p.n + blockIdx.y * 128 +
                                                  warp * 16 + j * 8 + t4 * 2) =
                        pack_bf16x2(acc[0][j][i * 2], acc[0][j][i * 2 + 1]);
    } else {
        float h[2][4];
        uint32_t m[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[j][i] = silu_mul(acc[0][j][i], acc[kHalves - 1][j][i]);
                m[i >> 1] = max(m[i >> 1], abs_bits(h[j][i]));
            }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[i] = max(m[i], __shfl_xor_sync(kFull, m[i], 1));
            m[i] = max(m[i], __shfl_xor_sync(kFull, m[i], 2));
            if (t4 == 0) wmax[warp][gid + i * 8] = m[i];
        }
        __syncthreads();
        const int I = p.n >> 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t am = 0;
            for (int w = 0; w < 8; ++w) am = max(am, wmax[w][gid + i * 8]);
            const float scale = block_scale(am);
            if (r0 + gid + i * 8 >= g.y) continue;
            const size_t row = row0 + gid + i * 8;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t c = scale == 0.0f ? 0u : code4(h[j][i * 2], h[j][i * 2 + 1], 0.0f, 0.0f, scale);
                *reinterpret_cast<uint16_t *>(p.h_q + row * I + blockIdx.y * 128 + warp * 16 + j * 8 + t4 * 2) = (uint16_t)c;
            }
            if (warp == 0 && t4 == 0) p.h_s[row * (I >> 7) + blockIdx.y] = scale;
        }
    }
}

static cudaError_t launch_product(const Product &p, cudaStream_t st) {
    if (p.cap == 0) return cudaSuccess;
    const unsigned tiles = (unsigned)((p.cap + 15) / 16);
    if (p.y)
        return launch_kernel(k_product_simple<false>, dim3(tiles, p.n >> 7, p.E), dim3(256), 0, st, p);
    return launch_kernel(k_product_simple<true>, dim3(tiles, p.n >> 8, p.E), dim3(256), 0, st, p);
}

// The checks that both products share; fills *p.
static int check_product(const moe_shape *sh, int64_t n, int k, const uint8_t *a_q,
                         const float *a_s, const int32_t *grp_off, const uint8_t *w_q,
                         const float *w_s, Product *p) {
    moe_sizes z;
    int rc = moe_sizes_query(sh, &z);
    if (rc != MOE_OK) return rc;
    if ((rc = check_width(n)) != MOE_OK || (rc = check_width(k)) != MOE_OK) return rc;
    const int64_t rows = (int64_t)sh->N * z.cap;
    if (!ok_buffer(a_q, rows * k) || !ok_buffer(a_s, rows * (k / 128) * 4) ||
        !ok_buffer(w_q, sh->E * n * k) || !ok_buffer(w_s, 4) || !ok_optional(grp_off))
        return MOE_EINVAL;
    if (!grp_off && sh->E != sh->N) return MOE_EINVAL;
    *p = Product{sh->N, sh->E, (int)z.cap, (int)n, k, a_q, a_s, grp_off, w_q, w_s, nullptr, nullptr, nullptr};
    return MOE_OK;
}

}  // namespace moe

extern "C" int moe_expert_gemm(const moe_shape *sh, int n, int k, const uint8_t *a_q,
                               const float *a_s, const int32_t *grp_off, const uint8_t *w_q,
                               const float *w_s, uint16_t *y, void *stream) {
    MOE_TRACE_CALL();
    moe::Product p;
    const int rc = moe::check_product(sh, n, k, a_q, a_s, grp_off, w_q, w_s, &p);
    if (rc != MOE_OK) return rc;
    if (!moe::ok_buffer(y, (int64_t)p.N * p.cap * n * 2)) return MOE_EINVAL;
    if (p.cap == 0) return MOE_OK;
    p.y = y;
    return moe::launch_product(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                       : MOE_ECUDA;
}

extern "C" int moe_expert_gemm_swiglu(const moe_shape *sh, int inter, int k, const uint8_t *a_q,
                                      const float *a_s, const int32_t *grp_off,
                                      const uint8_t *w13_q, const float *w13_s, uint8_t *h_q,
                                      float *h_s, void *stream) {
    MOE_TRACE_CALL();
    moe::Product p;
    int rc = moe::check_width(inter);
    if (rc != MOE_OK) return rc;
    rc = moe::check_product(sh, 2 * (int64_t)inter, k, a_q, a_s, grp_off, w13_q, w13_s, &p);
    if (rc != MOE_OK) return rc;
    const int64_t rows = (int64_t)p.N * p.cap;
    if (!moe::ok_buffer(h_q, rows * inter) || !moe::ok_buffer(h_s, rows * (inter / 128) * 4))
        return MOE_EINVAL;
    if (p.cap == 0) return MOE_OK;
    p.h_q = h_q;
    p.h_s = h_s;
    return moe::launch_product(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                       : MOE_ECUDA;
}
