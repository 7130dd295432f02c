// block.cu -- moe_block_norm: the norm after a branch, its gate and scale, the
// residual addition, the next norm and its block-128 e4m3 coding in one pass.
//
// A row stays with its CTA, as it was read, through both sums of squares: HBM is read and
// written once.  It stays in registers, but for what the compiler spills: 24 bytes a thread
// where 32 registers hold two chunks (the way of 7168), 320 where 64 hold eight (rows
// wider than 32768).  Measured with every input and output: 32767 rows of 7168 308 us (6.9
// TB/s, as much as a copy), 2048 rows 26 with bf16 out only (4.5 TB/s: a batch of 2048 is
// 3.4 rounds of CTAs, and each waits for its loads and two sums), one row 3.2.  Vectors
// come by plain loads: through the read-only path, which is not for what the kernel before
// may write, the compiler held more of them at once and spilled 64 bytes (323 us).
// Slower when this took 332 to 392: rows by bulk copies one to three ahead in CTAs that stay
// (437 to 580 us), both sums in one round (425 to 444; v's square from x's, the products'
// and the residual's sums), 896 threads with a chunk each (476).
#include <cmath>

#include "bf16.cuh"
#include "check.h"
#include "coding.cuh"
#include "launch.h"
#include "tc.cuh"
#include "trace.h"

namespace moe {

struct BlockNorm {
    int H, rows;
    int ahead;  // rows from one's own to the one that is brought to L2 (kAhead)
    uint64_t gate_of;  // 2^64 / rows that share a row of gate, above it; 0: each has its own
    float eps, scale, inv_H;
    const uint16_t *x, *post, *gate, *res, *gamma;
    uint16_t *res_out, *y;
    uint8_t *q;
    float *s;
};

// The sum of one value a thread, over the block or over the warp; `part` is shared
// float[32], not in use by anyone else.
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float *part) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    if (kWarp) return v;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float sum = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    return sum;
}

__device__ __forceinline__ uint4 vec8(const uint16_t *p, int c) {
    return *reinterpret_cast<const uint4 *>(p + c * 8);
}

// Eight bf16 values as four pairs of floats; pairs keep the instructions few, which
// bound this kernel with its threads.
__device__ __forceinline__ void widen8(uint64_t (&v)[4], const uint4 &w) {
    v[0] = widen2(w.x), v[1] = widen2(w.y), v[2] = widen2(w.z), v[3] = widen2(w.w);
}
__device__ __forceinline__ uint32_t narrow2(uint64_t v) {
    const float2 f = unpack2(v);
    return pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ uint4 narrow8(const uint64_t (&v)[4]) {
    return make_uint4(narrow2(v[0]), narrow2(v[1]), narrow2(v[2]), narrow2(v[3]));
}
__device__ __forceinline__ uint64_t both(float f) {
    return pack2(__float_as_uint(f), __float_as_uint(f));
}
__device__ __forceinline__ float sum2(uint64_t v) {
    const float2 f = unpack2(v);
    return f.x + f.y;
}

// A row, the block's or (kWarp) the warp's, from its V chunks of eight elements a
// thread, chunk tid + i * nthr of them: xr holds x, r the residual, as they were read:
// unpacked they would take twice the registers while the first sum is waited for.
template <int V, bool kWarp>
__device__ __forceinline__ void row_norm(const BlockNorm &p, size_t row, const uint4 (&xr)[V],
                                         const uint4 (&r)[V], float *part0, float *part1) {
    const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x, nthr = kWarp ? 32 : blockDim.x;
    const int nch = p.H >> 3;
    const size_t base = row * (size_t)p.H;
    float rstd = 1.0f;
    uint64_t acc = 0;
    if (p.post) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (tid + i * nthr < nch) {
                uint64_t w[4];
                widen8(w, xr[i]);
#pragma unroll
                for (int u = 0; u < 4; ++u) acc = fma2(w[u], w[u], acc);
            }
        rstd = rsqrtf(row_sum<kWarp>(sum2(acc), part0) * p.inv_H + p.eps);
        acc = 0;
    }
    uint64_t v[V][4];
    const uint16_t *gate = p.gate;
    if (gate) gate += (p.gate_of ? __umul64hi(row, p.gate_of) : row) * p.H;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * nthr;
        if (c >= nch) continue;
        uint64_t w[4];
        widen8(v[i], xr[i]);
        if (p.post) {
            widen8(w, vec8(p.post, c));
#pragma unroll
            for (int u = 0; u < 4; ++u) v[i][u] = mul2(mul2(v[i][u], both(rstd)), w[u]);
        }
        if (gate) {
            widen8(w, vec8(gate, c));
#pragma unroll
            for (int u = 0; u < 4; ++u) v[i][u] = mul2(v[i][u], w[u]);
        }
        widen8(w, r[i]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            v[i][u] = fma2(both(p.scale), v[i][u], w[u]);
            acc = fma2(v[i][u], v[i][u], acc);
        }
        if (p.res_out) *reinterpret_cast<uint4 *>(p.res_out + base + c * 8) = narrow8(v[i]);
    }
    if (!p.y && !p.q) return;
    rstd = rsqrtf(row_sum<kWarp>(sum2(acc), part1) * p.inv_H + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * nthr;
        const bool in = c < nch;
        uint32_t amax = 0;
        float f[8];
        if (in) {
            uint64_t w[4];
            widen8(w, vec8(p.gamma, c));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[i][u] = mul2(mul2(v[i][u], both(rstd)), w[u]);
                const float2 g = unpack2(v[i][u]);
                f[2 * u] = g.x, f[2 * u + 1] = g.y;
            }
            if (p.y) *reinterpret_cast<uint4 *>(p.y + base + c * 8) = narrow8(v[i]);
            amax = amax8(f);
        }
        if (p.q) {
            // the sixteen chunks of a block of 128 are sixteen neighbouring lanes
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) amax = max(amax, __shfl_xor_sync(kFull, amax, d));
            if (in) {
                const float scale = block_scale(amax);
                *reinterpret_cast<uint2 *>(p.q + base + c * 8) = code8_by(f, scale);
                if ((c & 15) == 0) p.s[row * (size_t)(p.H >> 7) + (c >> 4)] = scale;
            }
        }
    }
}

// `bytes` from p on, both multiples of 16, to L2.
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// One CTA per row, or one warp for short ones.
constexpr int kRowWarps = 4;
template <int V, int kMost, bool kWarp, bool kAhead>
__global__ void __launch_bounds__(kMost, kMost == 512 ? (V <= 2 ? 4 : V == 4 ? 2 : 1) : 1)
    k_block_norm(const __grid_constant__ BlockNorm p) {
    __shared__ float part[2][32];
    const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x, nthr = kWarp ? 32 : blockDim.x;
    const int nch = p.H >> 3;
    const size_t row = kWarp ? (size_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
    const size_t base = row * (size_t)p.H;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (kWarp && row >= p.rows) return;
    uint4 x[V], r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * nthr;
        x[i] = r[i] = make_uint4(0, 0, 0, 0);
        if (c >= nch) continue;
        x[i] = *reinterpret_cast<const uint4 *>(p.x + base + c * 8);
        if (p.res) r[i] = *reinterpret_cast<const uint4 *>(p.res + base + c * 8);
    }
    if (kAhead && tid == 0 && row + p.ahead < p.rows) {
        const size_t next = base + (size_t)p.ahead * p.H;
        prefetch_l2(p.x + next, 2 * p.H);
        if (p.res) prefetch_l2(p.res + next, 2 * p.H);
    }
    row_norm<V, kWarp>(p, row, x, r, part[0], part[1]);
}

template <class K>
static cudaError_t launch(K kern, int grid, int threads, const BlockNorm &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

static cudaError_t launch_block_norm(BlockNorm p, cudaStream_t st) {
    const int nch = p.H >> 3, rows = p.rows, sms = sm_count();
    if (rows > 2 * sms && nch <= 64) {
        const auto kern =
            nch <= 32 ? k_block_norm<1, 128, true, false> : k_block_norm<2, 128, true, false>;
        return launch(kern, (rows + kRowWarps - 1) / kRowWarps, 32 * kRowWarps, p, st);
    }
    const int most = rows <= sms ? 1024 : 512;
    int V = rows > 2 * sms ? 2 : 1;
    while (V < 8 && nch > most * V) V *= 2;
    const int nthr = ((nch + V - 1) / V + 31) / 32 * 32;
    // CTAs of rows wider than 4096 leave warps of an SM without work, and their loads wait:
    // each brings a later row to L2.  us without and with it: 32767 rows of 7168 325 and 308, of
    // 4096 177 and 175; 8192 of 4608 57.1 and 55.8, of 8192 95 and 92, of 12288 164 and 150; 2048
    // of 7168 25.2 and 24.2.  Rows four times as far ahead, and farther: 330 to 420.
    p.ahead = sms;
    const auto kern = nthr <= 512 ? (V == 1     ? k_block_norm<1, 512, false, false>
                                     : nch <= 512 ? k_block_norm<2, 512, false, false>
                                     : V == 2   ? k_block_norm<2, 512, false, true>
                                     : V == 4   ? k_block_norm<4, 512, false, true>
                                                : k_block_norm<8, 512, false, true>)
                                  : (V == 1   ? k_block_norm<1, 1024, false, false>
                                     : V == 2 ? k_block_norm<2, 1024, false, false>
                                     : V == 4 ? k_block_norm<4, 1024, false, false>
                                              : k_block_norm<8, 1024, false, false>);
    return launch(kern, rows, nthr, p, st);
}

}  // namespace moe

extern "C" int moe_block_norm(const moe_shape *sh, float eps, float scale, int gates,
                              const uint16_t *x, const uint16_t *post, const uint16_t *gate,
                              const uint16_t *res, const uint16_t *gamma, uint16_t *res_out,
                              uint16_t *y, uint8_t *q, float *s, void *stream) {
    MOE_TRACE_CALL();
    moe_sizes z;
    const int rc = moe_sizes_query(sh, &z);
    if (rc != MOE_OK) return rc;
    if (!(eps >= 0.0f) || std::isinf(eps) || !std::isfinite(scale)) return MOE_EINVAL;
    if (!moe::ok_optional(post) || !moe::ok_optional(gate) || !moe::ok_optional(res) ||
        !moe::ok_optional(gamma) || !moe::ok_optional(res_out) || !moe::ok_optional(y) ||
        !moe::ok_optional(q) || !moe::ok_optional(s))
        return MOE_EINVAL;
    const int64_t rows = (int64_t)sh->N * sh->T;
    if (gate && (gates < 1 || rows % gates != 0)) return MOE_EINVAL;
    if (rows == 0) return MOE_OK;
    if ((q == nullptr) != (s == nullptr) || (!res_out && !y && !q)) return MOE_EINVAL;
    if (!moe::ok_buffer(x, z.bytes_x) || ((y || q) && !gamma)) return MOE_EINVAL;
    if (rows >= ((int64_t)1 << 31)) return MOE_ENOTSUP;
    moe::BlockNorm p = {};
    p.H = sh->H;
    p.rows = (int)rows;
    if (gate && gates < rows) p.gate_of = ~0ull / (uint64_t)(rows / gates) + 1;
    p.inv_H = 1.0f / (float)sh->H;
    p.eps = eps;
    p.scale = scale;
    p.x = x;
    p.post = post;
    p.gate = gate;
    p.res = res;
    p.gamma = gamma;
    p.res_out = res_out;
    p.y = y;
    p.q = q;
    p.s = s;
    return moe::launch_block_norm(p, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ECUDA;
}
