// norm.cu -- moe_rmsnorm: residual addition, RMS norm and block-128 e4m3
// coding of the rows of x in one pass.
#include <cmath>

#include "bf16.cuh"
#include "check.h"
#include "coding.cuh"
#include "launch.h"
#include "trace.h"

namespace moe {

// One CTA per row.  A thread holds V chunks of eight elements in registers
// from the load to the last store, chunk tid + i * blockDim.x, so a row is
// read once; blockDim.x is a multiple of 32, so the sixteen chunks of a block
// of 128 are sixteen neighbouring lanes.
//
// Bound by HBM: per row 2 H bytes each of x, res, res_out and y and H (1 + 1/32)
// of codes.  With all of them, 32767 rows of 7168 take 309 us, 6.86 TB/s, as
// much as a copy.  What that took is threads in flight, not bytes a thread: two
// chunks a thread (448 threads a row) in 32 registers, four CTAs an SM; at 40
// registers and three CTAs 339 us, with four chunks a thread 379, eight 506.
// gamma is read again for the second half (L1 holds it) rather than kept in
// registers: 322 us with it kept.  Few rows have an SM each: one chunk a thread.
// The exact divisions of the coding are not what bounds it (379 us either way
// at four chunks), but their registers are.
constexpr int norm_ctas(int V, int most) { return most == 512 ? (V <= 2 ? 4 : V == 4 ? 2 : 1) : 1; }

template <int V, int kMost>
__global__ void __launch_bounds__(kMost, norm_ctas(V, kMost)) k_rmsnorm(int H, float eps, const uint16_t *x,
                                                   const uint16_t *res, const uint16_t *gamma,
                                                   uint16_t *res_out, uint16_t *y,
                                                   uint8_t *__restrict__ q, float *__restrict__ s) {
    __shared__ float wsum[32];
    const int tid = threadIdx.x, nthr = blockDim.x, nch = H >> 3;
    const size_t row = blockIdx.x, base = row * (size_t)H;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v[V][8], acc = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * nthr;
        if (c >= nch) continue;
        unpack8(v[i], *reinterpret_cast<const uint4 *>(x + base + c * 8));
        if (res) add8(v[i], *reinterpret_cast<const uint4 *>(res + base + c * 8));
#pragma unroll
        for (int u = 0; u < 8; ++u) acc = __fmaf_rn(v[i][u], v[i][u], acc);
    }
    if (res_out) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = tid + i * nthr;
            if (c < nch) *reinterpret_cast<uint4 *>(res_out + base + c * 8) = pack_bf16x8(v[i]);
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(kFull, acc, d);
    if ((tid & 31) == 0) wsum[tid >> 5] = acc;
    __syncthreads();
    float sum = (tid & 31) < (nthr >> 5) ? wsum[tid & 31] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    const float rstd = __frsqrt_rn(sum / (float)H + eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * nthr;
        const bool in = c < nch;
        uint32_t amax = 0;
        if (in) {
            float w[8];
            unpack8(w, *reinterpret_cast<const uint4 *>(gamma + c * 8));
#pragma unroll
            for (int u = 0; u < 8; ++u) v[i][u] = (v[i][u] * rstd) * w[u];
            if (y) *reinterpret_cast<uint4 *>(y + base + c * 8) = pack_bf16x8(v[i]);
            amax = amax8(v[i]);
        }
        if (q) {
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) amax = max(amax, __shfl_xor_sync(kFull, amax, d));
            if (in) {
                const float scale = block_scale(amax);
                *reinterpret_cast<uint2 *>(q + base + c * 8) = code8_by(v[i], scale);
                if ((c & 15) == 0) s[row * (size_t)(H >> 7) + (c >> 4)] = scale;
            }
        }
    }
}

template <int V, int kMost>
static cudaError_t launch_rows(int rows, int nthr, cudaStream_t st, int H, float eps,
                               const uint16_t *x, const uint16_t *res, const uint16_t *gamma,
                               uint16_t *res_out, uint16_t *y, uint8_t *q, float *s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)rows);
    cfg.blockDim = dim3((unsigned)nthr);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rmsnorm<V, kMost>, H, eps, x, res, gamma, res_out, y, q, s);
}

static cudaError_t launch_rmsnorm(const moe_shape &sh, float eps, const uint16_t *x,
                                  const uint16_t *res, const uint16_t *gamma, uint16_t *res_out,
                                  uint16_t *y, uint8_t *q, float *s, cudaStream_t st) {
    const int rows = sh.N * sh.T, nch = sh.H >> 3;
    const int most = rows <= sm_count() ? 1024 : 512;
    int V = 1;
    while (V < 8 && nch > most * V) V *= 2;
    const int nthr = ((nch + V - 1) / V + 31) / 32 * 32;
    const auto go = nthr <= 512
                        ? (V == 1   ? launch_rows<1, 512>
                           : V == 2 ? launch_rows<2, 512>
                           : V == 4 ? launch_rows<4, 512>
                                    : launch_rows<8, 512>)
                        : (V == 1   ? launch_rows<1, 1024>
                           : V == 2 ? launch_rows<2, 1024>
                           : V == 4 ? launch_rows<4, 1024>
                                    : launch_rows<8, 1024>);
    return go(rows, nthr, st, sh.H, eps, x, res, gamma, res_out, y, q, s);
}

}  // namespace moe

extern "C" int moe_rmsnorm(const moe_shape *sh, float eps, const uint16_t *x, const uint16_t *res,
                           const uint16_t *gamma, uint16_t *res_out, uint16_t *y, uint8_t *q,
                           float *s, void *stream) {
    MOE_TRACE_CALL();
    moe_sizes z;
    int rc = moe_sizes_query(sh, &z);
    if (rc != MOE_OK) return rc;
    if (!(eps >= 0.0f) || std::isinf(eps)) return MOE_EINVAL;
    if ((int64_t)sh->N * sh->T == 0) return MOE_OK;
    if ((q == nullptr) != (s == nullptr) || (!res_out && !y && !q)) return MOE_EINVAL;
    if (!moe::ok_buffer(x, z.bytes_x) || !moe::ok_buffer(gamma, 2 * sh->H) ||
        !moe::ok_optional(res) || !moe::ok_optional(res_out) || !moe::ok_optional(y) ||
        !moe::ok_optional(q) || !moe::ok_optional(s))
        return MOE_EINVAL;
    if ((int64_t)sh->N * sh->T >= ((int64_t)1 << 31)) return MOE_ENOTSUP;
    return moe::launch_rmsnorm(*sh, eps, x, res, gamma, res_out, y, q, s,
                               reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ECUDA;
}
