// topk.cu -- moe_topk: a router's choice of experts and their weights from logits.
//
// A warp has a token: its logits lie in the lanes' registers, lane l holding experts
// l * 4 .. l * 4 + 3 of every 128.  What chooses is turned into 32-bit integers
// whose order is the values', and the R largest are taken one after another by the
// warp's integer maximum.
//
// Without a bias the integers are the logits themselves, exactly.  With one, c = s +
// bias comes from fp32 and may be kCloseUlps off: where two neighbours among the
// first R + 1 (or the kept runs' worths) are closer than both errors, the token's
// candidates are evaluated and ordered again in 64 bits (about one token in a
// thousand at 256 experts; all of it in 64 bits would take the GPU's fp64 units 30
// times as long as the logits take to arrive).
#include <cmath>

#include "check.h"
#include "common.cuh"
#include "launch.h"
#include "trace.h"

namespace moe {

struct Router {
    int rows, E, R, score, groups, kept, best, renorm, per;
    unsigned per_inv;  // floor(e / per) == (e * per_inv) >> 20 for e < 1024
    float scale;
    const float *logits, *bias;
    int32_t *idx;
    float *w;
};

// Order-preserving integers of floats: larger for larger, the two zeros alike;
// kLowest for -infinity and NaN.  0 is left for "not there".
constexpr uint32_t kLowest = 0x007fffffu;
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return v == v ? k : kLowest;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// How far fp32's c (or sum of two) is from the 64-bit one, by its magnitude: the
// exponential's argument and result, the quotient and the sum of exponentials are
// less than 6 * 2^-24 of a score of at most 1 together, the addition 2^-24 of c.
__device__ __forceinline__ float error_of(float c) {
    return 0x1p-20f + fabsf(c) * 0x1p-22f;
}

__device__ __forceinline__ float score32(int score, float l, float top, float inv_sum) {
    return score == MOE_SCORE_SIGMOID ? 1.0f / (1.0f + expf(-l)) : expf(l - top) * inv_sum;
}

// The run of expert e, of E or of the padding behind them.
__device__ __forceinline__ int run_of(const Router &p, int e) {
    return min((int)((e * p.per_inv) >> 20), 31);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// Experts a lane holds, and the tokens of a CTA by it: shared memory bounds them.
__host__ __device__ constexpr int topk_warps(int C) { return C <= 16 ? 4 : 2; }

// A warp's part of the 64-bit evaluation.
template <int C>
struct Exact {
    double c[C * 32];
    uint16_t list[C * 32];
};

// An expert's c (its score without a bias) in 64 bits.
__device__ __forceinline__ double value64(const Router &p, const float *l, int e, float top,
                                          double sum) {
    const float v = l[e];
    double c = p.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-(double)v))
                                            : exp((double)v - (double)top) / sum;
    if (p.bias) c += (double)p.bias[e];
    return v != -INFINITY && c == c ? c : -(double)INFINITY;
}

__device__ __forceinline__ double sum64(const Router &p, const float *l, float top) {
    if (p.score == MOE_SCORE_SIGMOID) return 1.0;
    double sum = 0.0;
    for (int e = threadIdx.x & 31; e < p.E; e += 32) sum += exp((double)l[e] - (double)top);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    return sum;
}

// The kept runs in 64 bits, one bit each, by all lanes of a warp.
__device__ __noinline__ uint32_t kept64(const Router &p, const float *l, double *c, float top) {
    const int lane = threadIdx.x & 31;
    const double sum = sum64(p, l, top);
    for (int e = lane; e < p.E; e += 32) c[e] = value64(p, l, e, top, sum);
    __syncwarp();
    double worth = -(double)INFINITY;
    if (lane < p.groups) {
        double a = worth, b = worth;  // the two largest
        for (int e = lane * p.per; e < (lane + 1) * p.per; ++e) {
            b = fmax(b, fmin(a, c[e]));
            a = fmax(a, c[e]);
        }
        worth = p.best == 2 ? a + b : a;
    }
    int before = 0;
    for (int g = 0; g < p.groups; ++g) {
        const double o = __shfl_sync(kFull, worth, g);
        before += o > worth || (o == worth && g < lane);
    }
    __syncwarp();
    return __ballot_sync(kFull, lane < p.groups && before < p.kept);
}

// The choice in 64 bits, by all lanes of a warp, of the kept experts whose c is
// `least` or more in fp32: lane r gets the r-th.  Only with a bias.
__device__ __noinline__ int choose64(const Router &p, const float *l, double *c, uint16_t *list,
                                     float top, uint32_t kept, float least) {
    const int lane = threadIdx.x & 31;
    const double sum = sum64(p, l, top);
    int n = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {  // listed in the order of their index
        const int e = e0 + lane;
        bool in = e < p.E && (kept >> run_of(p, e) & 1u);
        if (in) {
            const float v = l[e];
            float c = score32(p.score, v, top, (float)(1.0 / sum)) + p.bias[e];
            if (v == -INFINITY || c != c) c = -INFINITY;
            in = c >= least;
        }
        const unsigned who = __ballot_sync(kFull, in);
        if (in) list[n + __popc(who & ((1u << lane) - 1u))] = (uint16_t)e;
        n += __popc(who);
    }
    __syncwarp();
    for (int j = lane; j < n; j += 32) c[j] = value64(p, l, list[j], top, sum);
    __syncwarp();
    int mine = 0;
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        int before = 32;
        if (j < n) {
            before = 0;
            for (int o = 0; o < n; ++o) before += c[o] > c[j] || (c[o] == c[j] && o < j);
        }
        for (int o = 0; o < 32; ++o)  // candidate j0 + o goes to the lane of its rank
            if (__shfl_sync(kFull, before, o) == lane) mine = list[j0 + o];
    }
    return mine;
}

template <int C>
__global__ void __launch_bounds__(32 * topk_warps(C)) k_topk(const Router p) {
    constexpr int kWarps = topk_warps(C);
    __shared__ Exact<C> exact[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row = blockIdx.x * kWarps + warp;
    if (row >= p.rows) return;
    const float *l = p.logits + (size_t)row * p.E;
    // v[4 q + j]: expert 128 q + 4 lane + j
    float v[C];
    const bool quads = (p.E & 3) == 0;  // then every row starts on 16 bytes
#pragma unroll
    for (int q = 0; q < (C + 3) / 4; ++q) {
        const int e = q * 128 + lane * 4;
        if (quads) {
            float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e < p.E) f = __ldg(reinterpret_cast<const float4 *>(l + e));
            v[4 * q] = f.x;
            v[4 * q + 1] = f.y;
            v[4 * q + 2] = f.z;
            v[4 * q + 3] = f.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * q + j] = e + j < p.E ? __ldg(l + e + j) : -INFINITY;
        }
    }
    const auto expert = [&](int i) { return (i >> 2) * 128 + lane * 4 + (i & 3); };
    bool bad = false;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        bad |= v[i] != v[i] || (p.score == MOE_SCORE_SOFTMAX && v[i] == INFINITY);
        top = fmaxf(top, v[i]);
    }
    bad = __any_sync(kFull, bad);
    top = warp_max(top);
    // the sum of the exponentials, where a value needs it
    const bool scores = p.bias || (p.groups > 1 && p.best == 2);
    float inv_sum = 1.0f;
    if (p.score == MOE_SCORE_SOFTMAX && (scores || !p.renorm)) {
        float sum = 0.0f;
        if (top > -INFINITY)
#pragma unroll
            for (int i = 0; i < C; ++i) sum += expf(v[i] - top);
        sum = warp_sum(sum);
        inv_sum = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    // what is compared: c, or the logits; masked experts last, the padding not there
    uint32_t key[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = expert(i);
        float c = v[i];
        if (p.bias && e < p.E && v[i] != -INFINITY)
            c = score32(p.score, v[i], top, inv_sum) + __ldg(p.bias + e);
        key[i] = e < p.E ? key_of(c) : 0u;
    }
    // the kept runs
    uint32_t kept = 0xffffffffu;
    if (p.groups > p.kept) {
        float slack = 0.0f;  // both errors of two runs' worths
        uint32_t mine = 0;  // lane g: the worth of run g
        for (int g = 0; g < p.groups; ++g) {
            uint32_t a = 0, b = 0;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (run_of(p, expert(i)) != g) continue;
                uint32_t k = key[i];
                if (!p.bias && p.best == 2 && k > kLowest)
                    k = key_of(score32(p.score, v[i], top, inv_sum));
                b = max(b, min(a, k));
                a = max(a, k);
            }
            const uint32_t first = __reduce_max_sync(kFull, a);
            uint32_t worth = first;
            float error = error_of(value_of(first));
            if (p.best == 2) {
                const unsigned who = __ballot_sync(kFull, a == first);
                // the second largest: the others' first, or this lane's second
                const uint32_t rest = (who & (who - 1)) || a != first ? a : b;
                const uint32_t second = __reduce_max_sync(kFull, rest);
                worth = key_of(value_of(first) + value_of(second));
                error += error_of(value_of(second));
            }
            if (worth > kLowest) slack = fmaxf(slack, 2.0f * error);
            if (lane == g) mine = worth;
        }
        int before = 0;
        for (int g = 0; g < p.groups; ++g) {
            const uint32_t o = __shfl_sync(kFull, mine, g);
            before += o > mine || (o == mine && g < lane);
        }
        const bool run = lane < p.groups;
        kept = __ballot_sync(kFull, run && before < p.kept);
        if (p.bias || p.best == 2) {
            // the least kept and the best of the others
            const uint32_t in = __reduce_min_sync(kFull, run && before < p.kept ? mine : ~0u);
            const uint32_t out = __reduce_max_sync(kFull, run && before >= p.kept ? mine : 0u);
            if (out > kLowest && value_of(in) - value_of(out) <= slack)
                kept = kept64(p, l, exact[warp].c, top);
        }
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (!(kept >> run_of(p, expert(i)) & 1u)) key[i] = 0u;
    }
    // the R largest, and with a bias the one behind them
    int mine = 0;
    bool close = false;
    uint32_t last = ~0u;
    const int rounds = p.bias ? p.R + 1 : p.R;
    for (int r = 0; r < rounds; ++r) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) m = max(m, key[i]);
        const uint32_t most = __reduce_max_sync(kFull, m);
        if (most == 0u) break;  // no one is behind the R
        if (p.bias && last != ~0u) {
            const float a = value_of(last), b = value_of(most);
            close |= b > -INFINITY && a - b <= error_of(a) + error_of(b);
        }
        last = most;
        int at = 0x10000;
#pragma unroll
        for (int i = C - 1; i >= 0; --i)
            if (key[i] == most) at = expert(i);
        const int e = (int)__reduce_min_sync(kFull, (unsigned)at);
        if (r == p.R) break;
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (expert(i) == e) key[i] = 0u;
        if (lane == r) mine = e;
    }
    if (close) {
        // nothing below the last one by more than both errors can be among the first R
        const float c = value_of(last);
        mine = choose64(p, l, exact[warp].c, exact[warp].list, top, kept,
                        c > -INFINITY ? c - 2.0f * error_of(c) : -INFINITY);
    }
    // the weights, lane r the r-th
    const bool chosen = lane < p.R;
    const float lv = chosen ? __ldg(l + mine) : -INFINITY;
    float s = 0.0f;
    if (p.renorm) {
        // all of them times exp(-m), so that small ones keep their ratios
        const float m = warp_max(lv);
        if (lv > -INFINITY)
            s = p.score == MOE_SCORE_SOFTMAX ? expf(lv - m)
                : m >= 0.0f                  ? score32(p.score, lv, top, inv_sum)
                                             : expf(lv - m) / (1.0f + expf(lv));
        const float sum = warp_sum(s);
        s = sum > 0.0f ? s / sum : 0.0f;
    } else if (lv > -INFINITY) {
        s = score32(p.score, lv, top, inv_sum);
    }
    if (chosen) {
        p.idx[(size_t)row * p.R + lane] = mine;
        p.w[(size_t)row * p.R + lane] = bad ? __uint_as_float(0x7fffffffu) : s * p.scale;
    }
}

template <int C>
static cudaError_t launch(const Router &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((p.rows + topk_warps(C) - 1) / topk_warps(C)));
    cfg.blockDim = dim3(32 * topk_warps(C));
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_topk<C>, p);
}

static cudaError_t launch_topk(const Router &p, cudaStream_t st) {
    if (p.E <= 128) return launch<4>(p, st);
    if (p.E <= 256) return launch<8>(p, st);
    if (p.E <= 512) return launch<16>(p, st);
    return launch<32>(p, st);
}

}  // namespace moe

extern "C" int moe_topk(const moe_shape *sh, int score, int groups, int kept, int best, int renorm,
                        float scale, const float *logits, const float *bias, int32_t *topk_idx,
                        float *topk_w, void *stream) {
    MOE_TRACE_CALL();
    moe_sizes z;
    const int rc = moe_sizes_query(sh, &z);
    if (rc != MOE_OK) return rc;
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
    if (groups < 1 || sh->E % groups != 0 || kept < 1 || kept > groups || !std::isfinite(scale))
        return MOE_EINVAL;
    const int per = sh->E / groups;
    if (best < 1 || best > 2 || best > per || sh->R > kept * per) return MOE_EINVAL;
    if (groups > MOE_MAX_GROUPS) return MOE_ENOTSUP;
    const int64_t rows = (int64_t)sh->N * sh->T;
    if (!moe::ok_buffer(logits, rows * sh->E * 4) || !moe::ok_optional(bias) ||
        !moe::ok_buffer(topk_idx, z.bytes_topk_idx) || !moe::ok_buffer(topk_w, z.bytes_topk_idx))
        return MOE_EINVAL;
    if (rows == 0) return MOE_OK;
    if (rows >= ((int64_t)1 << 31) - 4) return MOE_ENOTSUP;
    const unsigned inv = ((1u << 20) + per - 1) / per;
    const moe::Router p = {(int)rows, sh->E,  sh->R, score,  groups, kept,     best,  renorm != 0,
                           per,       inv,    scale, logits, bias,   topk_idx, topk_w};
    return moe::launch_topk(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                      : MOE_ECUDA;
}
