// few.cu -- moe_layer_few: a whole expert layer for a few tokens in two
// kernels, bound by reading the chosen experts' weights once.
//
// k_few_up reads the gate and up weights of each chosen expert and leaves the
// coded activations h of every (token, expert) pair; k_few_down reads the
// down weights and leaves each token's weighted sum.  Both hand the weights
// to the tensor cores as the 16-row operand of mma.m16n8k32 straight from
// global memory, with up to eight tokens as the 8-column operand: a weight
// byte is loaded once, is never converted, and meets its tokens in one
// instruction, so the product costs less than its loads (a warp issues four
// MMAs for every four 512-byte loads) and the kernels are bound by HBM.
// tcgen05 would stage the same bytes through shared memory for a 128-row tile
// that a few tokens cannot fill.
//
// The k order within a block of 128 is permuted, alike for both operands: a
// lane loads 16 consecutive bytes of its row (four lanes of a row 64) and
// feeds words 0 and 1 to one MMA and words 2 and 3 to the next.
#include <cooperative_groups.h>

#include "bf16.cuh"
#include "check.h"
#include "coding.cuh"
#include "launch.h"
#include "mma8.cuh"
#include "trace.h"

namespace moe {

namespace cg = cooperative_groups;

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewCluster = 8;  // CTAs that share one block of 128 activations

struct Few {
    int ntok, E, R, H, inter;
    int per;  // tokens whose coded x fits a CTA's shared memory at once, at most 8
    const uint16_t *x;
    const int32_t *idx;
    const float *topk_w;
    const uint8_t *w13_q;
    const float *w13_s;
    const uint8_t *w2_q;
    const float *w2_s;
    uint8_t *h_q;
    float *h_s;
    uint16_t *out;
    int32_t *status;
};

// Two rows (g and g + 8 of a 16-row tile) of one block of 128 along k: lane
// (g, t) holds bytes 16 t .. 16 t + 15 of each half of 64.
struct Tile16 {
    uint4 lo[2], hi[2];  // [half]: row g, row g + 8
};

__device__ __forceinline__ void load_tile(Tile16 &w, const uint8_t *row_g, size_t pitch8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w.lo[i] = __ldcs(reinterpret_cast<const uint4 *>(row_g + i * 64));
        w.hi[i] = __ldcs(reinterpret_cast<const uint4 *>(row_g + pitch8 + i * 64));
    }
}

// c = tile times the column operand x (words as load_tile's), one block of 128.
__device__ __forceinline__ void mma_tile(float (&c)[4], const Tile16 &w, const uint4 (&x)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a0[4] = {w.lo[i].x, w.hi[i].x, w.lo[i].y, w.hi[i].y};
        const uint32_t a1[4] = {w.lo[i].z, w.hi[i].z, w.lo[i].w, w.hi[i].w};
        mma_e4m3(c, a0, x[i].x, x[i].y);
        mma_e4m3(c, a1, x[i].z, x[i].w);
    }
}

// Row pitch of the coded x in shared memory: 64 bytes past a multiple of 128,
// so the two rows that eight lanes of a 16-byte load touch fall on different
// banks.
__host__ __device__ constexpr int few_pitch(int H) { return H + 64; }

__host__ __device__ constexpr size_t few_up_smem(int H, int m) {
    return (size_t)m * few_pitch(H) + (size_t)m * (H >> 7) * 4;
}

// A cluster of eight CTAs: one expert's block of 128 activations, CTA c the
// gate and up rows 16 c .. 16 c + 15 of it; its warps take the blocks along H
// in turn.  grid.z counts assignments: the cluster of an expert's first
// assignment works for all its tokens, eight at a time, the others return.
__global__ void __launch_bounds__(kFewThreads) __cluster_dims__(kFewCluster, 1, 1)
    k_few_up(const Few p) {
    extern __shared__ __align__(16) uint8_t few_smem[];
    __shared__ float red[kFewWarps][2][16][8];
    __shared__ uint32_t peak[2][kFewCluster][8];  // amax parts of all CTAs, by pass
    __shared__ int list[MOE_FEW_MAX_TOKENS];      // the expert's assignments, one a token
    __shared__ unsigned chosen[2];
    __shared__ __align__(16) uint8_t codes[8][16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int c = blockIdx.x, blk = blockIdx.y, a = blockIdx.z;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (c == 0 && blk == 0 && a == 0) {
        int bad = 0;
        for (int i = tid; i < p.ntok * p.R; i += kFewThreads)
            bad |= (unsigned)__ldg(p.idx + i) >= (unsigned)p.E;
        bad = __syncthreads_or(bad);
        if (tid == 0) *p.status = bad ? MOE_ST_BAD_EXPERT : 0;
    }
    const int e = __ldg(p.idx + a);
    if ((unsigned)e >= (unsigned)p.E) return;
    // thread t < 64: token t's first assignment to this expert
    if (tid < MOE_FEW_MAX_TOKENS) {
        int k = -1;
        if (tid < p.ntok)
            for (int i = p.R - 1; i >= 0; --i)
                if (__ldg(p.idx + tid * p.R + i) == e) k = i;
        const unsigned got = __ballot_sync(kFull, k >= 0);
        if (lane == 0) chosen[warp] = got;
        list[tid] = k;  // by token for now
    }
    __syncthreads();
    const unsigned lo = chosen[0], hi = chosen[1];
    const int first = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
    if (first * p.R + list[first] != a) return;  // an earlier assignment's cluster does it
    const int m = __popc(lo) + __popc(hi);
    {
        const int k = tid < MOE_FEW_MAX_TOKENS ? list[tid] : -1;
        __syncthreads();
        if (k >= 0) {
            const unsigned below = (1u << lane) - 1u;
            const int at = warp == 0 ? __popc(lo & below) : __popc(lo) + __popc(hi & below);
            list[at] = tid * p.R + k;
        }
        __syncthreads();
    }

    const int H = p.H, Hb = H >> 7, pitch = few_pitch(H), I = p.inter;
    float *xs = reinterpret_cast<float *>(few_smem + (size_t)p.per * pitch);
    const uint8_t *gate = p.w13_q + ((size_t)e * 2 * I + blk * 128 + c * 16 + g) * H + t4 * 16;
    const uint8_t *up = gate + (size_t)I * H;
    const float *gs = p.w13_s + ((size_t)e * 2 * (I >> 7) + blk) * Hb;
    const float *us = gs + (size_t)(I >> 7) * Hb;
    const size_t p8 = (size_t)8 * H;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();  // waited for before the first store to another CTA

    for (int n0 = 0, pass = 0; n0 < m; n0 += p.per, pass ^= 1) {
        const int mm = min(p.per, m - n0);
        // the first weights are on their way while x is coded
        Tile16 wg, wu;
        int b = warp;
        if (b < Hb) {
            load_tile(wg, gate + b * 128, p8);
            load_tile(wu, up + b * 128, p8);
        }
        for (int i = warp; i < mm * Hb; i += kFewWarps) {
            const int n = i / Hb, bb = i - n * Hb, tok = list[n0 + n] / p.R;
            const uint2 v = *reinterpret_cast<const uint2 *>(p.x + (size_t)tok * H + bb * 128 + lane * 4);
            const float f0 = bf16_lo(v.x), f1 = bf16_hi(v.x), f2 = bf16_lo(v.y), f3 = bf16_hi(v.y);
            const uint32_t am = __reduce_max_sync(
                kFull, max(max(abs_bits(f0), abs_bits(f1)), max(abs_bits(f2), abs_bits(f3))));
            const float scale = block_scale(am);
            *reinterpret_cast<uint32_t *>(few_smem + (size_t)n * pitch + bb * 128 + lane * 4) =
                scale == 0.0f ? 0u : code4(f0, f1, f2, f3, scale);
            if (lane == 0) xs[n * Hb + bb] = scale;
        }
        __syncthreads();
        // absent columns read a row that is there; their sums are dropped
        const uint8_t *xr = few_smem + (size_t)min(g, mm - 1) * pitch + t4 * 16;
        const float *s0 = xs + min(2 * t4, mm - 1) * Hb, *s1 = xs + min(2 * t4 + 1, mm - 1) * Hb;
        float ag[4] = {}, au[4] = {};
        for (; b < Hb; b += kFewWarps) {
            Tile16 ng, nu;
            const int nb = b + kFewWarps;
            if (nb < Hb) {
                load_tile(ng, gate + nb * 128, p8);
                load_tile(nu, up + nb * 128, p8);
            }
            const uint4 x[2] = {*reinterpret_cast<const uint4 *>(xr + b * 128),
                                *reinterpret_cast<const uint4 *>(xr + b * 128 + 64)};
            const float sg = __ldg(gs + b), su = __ldg(us + b), x0 = s0[b], x1 = s1[b];
            float cgt[4] = {}, cup[4] = {};
            mma_tile(cgt, wg, x);
            mma_tile(cup, wu, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ag[i] = __fmaf_rn(sg * ((i & 1) ? x1 : x0), cgt[i], ag[i]);
                au[i] = __fmaf_rn(su * ((i & 1) ? x1 : x0), cup[i], au[i]);
            }
            wg = ng;
            wu = nu;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            red[warp][0][g + 8 * (i >> 1)][2 * t4 + (i & 1)] = ag[i];
            red[warp][1][g + 8 * (i >> 1)][2 * t4 + (i & 1)] = au[i];
        }
        __syncthreads();
        if (n0 == 0) cluster.barrier_wait();
        // thread: token n = tid / 16, activation f = tid % 16 of this CTA
        float h = 0.0f;
        const int n = tid >> 4, f = tid & 15;
        if (tid < 128) {
            float vg = 0.0f, vu = 0.0f;
#pragma unroll
            for (int w = 0; w < kFewWarps; ++w) {
                vg += red[w][0][f][n];
                vu += red[w][1][f][n];
            }
            h = silu_mul(vg, vu);
            uint32_t am = abs_bits(h);
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) am = max(am, __shfl_xor_sync(kFull, am, d));
            // lane f < 8 tells CTA f of the cluster
            if (f < kFewCluster) *cluster.map_shared_rank(&peak[pass][c][n], f) = am;
        }
        cluster.sync();  // also orders the reads of red and x before their next use
        if (tid < 128) {
            uint32_t am = 0;
#pragma unroll
            for (int i = 0; i < kFewCluster; ++i) am = max(am, peak[pass][i][n]);
            const float scale = block_scale(am);
            codes[n][f] = scale == 0.0f ? 0 : (uint8_t)code4(h, 0.0f, 0.0f, 0.0f, scale);
            if (c == 0 && f == 0 && n < mm) p.h_s[(size_t)list[n0 + n] * (I >> 7) + blk] = scale;
            __syncwarp();
            if (f == 0 && n < mm)
                *reinterpret_cast<uint4 *>(p.h_q + (size_t)list[n0 + n] * I + blk * 128 + c * 16) =
                    *reinterpret_cast<const uint4 *>(codes[n]);
        }
    }
}

__host__ __device__ constexpr size_t few_down_smem(int ntok, int E, int R, int NT) {
    // ids, weights, first assignment of each expert, list of experts; sums
    return ((size_t)ntok * R * 2 + E * 2) * 4 + (size_t)kFewWarps * 16 * 8 * NT * 4;
}

// One CTA: 16 outputs of every token.  The (expert, block of 128 along
// inter) items are cut into eight equal runs, one a warp; the columns of the
// MMAs are the tokens themselves, so the sums over all experts stay in
// registers (NT tiles of eight tokens) with the routing weight in the scale.
template <int NT>
__global__ void __launch_bounds__(kFewThreads) k_few_down(const Few p) {
    extern __shared__ __align__(16) uint8_t few_smem[];
    const int A = p.ntok * p.R;
    float *red = reinterpret_cast<float *>(few_smem);  // [warp][16][8 NT]
    int *ids = reinterpret_cast<int *>(red + kFewWarps * 16 * 8 * NT);
    float *tw = reinterpret_cast<float *>(ids + A);
    int *head = reinterpret_cast<int *>(tw + A);  // [E] first assignment
    int *experts = head + p.E;                    // [U] in order of their heads
    __shared__ int wsum[32], total;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int f0 = blockIdx.x * 16, I = p.inter, Ib = I >> 7, H = p.H;

    for (int i = tid; i < p.E; i += kFewThreads) head[i] = A;
    __syncthreads();
    for (int i = tid; i < A; i += kFewThreads) {
        const int e = __ldg(p.idx + i);
        ids[i] = e;
        tw[i] = __ldg(p.topk_w + i);
        if ((unsigned)e < (unsigned)p.E) atomicMin(head + e, i);
    }
    __syncthreads();
    int U = 0;
    for (int i0 = 0; i0 < A; i0 += kFewThreads) {
        const int i = i0 + tid;
        const int e = i < A ? ids[i] : -1;
        const int is = (unsigned)e < (unsigned)p.E && head[e] == i;
        const int at = block_inclusive_scan(is, wsum, &total);
        if (is) experts[U + at - 1] = e;
        U += total;
        __syncthreads();
    }

    const int items = U * Ib;
    const int i0 = (int)((long long)items * warp / kFewWarps);
    const int i1 = (int)((long long)items * (warp + 1) / kFewWarps);
    const size_t p8 = (size_t)8 * I;
    const auto weights = [&](int item) {
        const int u = item / Ib;
        return p.w2_q + ((size_t)experts[u] * H + f0 + g) * I + (item - u * Ib) * 128 + t4 * 16;
    };
    float acc[NT][4] = {};
    Tile16 w;
    if (i0 < i1) load_tile(w, weights(i0), p8);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // h is k_few_up's

    int slot[NT];       // this lane's column token of each tile: its h row
    float rw[NT];       // and its routing weight
    unsigned on[NT];    // tokens of each tile that chose the expert
    int e = -1;
    for (int item = i0; item < i1; ++item) {
        const int u = item / Ib, b = item - u * Ib;
        Tile16 nw;
        if (item + 1 < i1) load_tile(nw, weights(item + 1), p8);
        if (e < 0 || b == 0) {
            e = experts[u];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int tok = t * 8 + g;
                slot[t] = -1;
                rw[t] = 0.0f;
                if (tok < p.ntok)
                    for (int k = 0; k < p.R; ++k)
                        if (ids[tok * p.R + k] == e) {
                            if (slot[t] < 0) slot[t] = tok * p.R + k;
                            rw[t] += tw[tok * p.R + k];
                        }
                on[t] = __ballot_sync(kFull, slot[t] >= 0);  // four equal bits a token
            }
        }
        const float ws = __ldg(p.w2_s + ((size_t)e * (H >> 7) + (f0 >> 7)) * Ib + b);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (on[t] == 0) continue;
            uint4 h[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            float fac = 0.0f;
            if (slot[t] >= 0) {
                const uint8_t *hr = p.h_q + (size_t)slot[t] * I + b * 128 + t4 * 16;
                h[0] = *reinterpret_cast<const uint4 *>(hr);
                h[1] = *reinterpret_cast<const uint4 *>(hr + 64);
                fac = rw[t] * p.h_s[(size_t)slot[t] * Ib + b];
            }
            float c[4] = {};
            mma_tile(c, w, h);
            const float c0 = ws * __shfl_sync(kFull, fac, 8 * t4);
            const float c1 = ws * __shfl_sync(kFull, fac, 8 * t4 + 4);
            // a token that did not choose the expert takes nothing of it, not
            // even 0 times a NaN weight
            if (on[t] >> (8 * t4) & 1u) {
                acc[t][0] = __fmaf_rn(c0, c[0], acc[t][0]);
                acc[t][2] = __fmaf_rn(c0, c[2], acc[t][2]);
            }
            if (on[t] >> (8 * t4 + 4) & 1u) {
                acc[t][1] = __fmaf_rn(c1, c[1], acc[t][1]);
                acc[t][3] = __fmaf_rn(c1, c[3], acc[t][3]);
            }
        }
        w = nw;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            red[(warp * 16 + g + 8 * (i >> 1)) * 8 * NT + t * 8 + 2 * t4 + (i & 1)] = acc[t][i];
    __syncthreads();
    for (int i = tid; i < p.ntok * 8; i += kFewThreads) {
        const int tok = i >> 3, f = (i & 7) * 2;
        float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
        for (int q = 0; q < kFewWarps; ++q) {
            v0 += red[(q * 16 + f) * 8 * NT + tok];
            v1 += red[(q * 16 + f + 1) * 8 * NT + tok];
        }
        *reinterpret_cast<uint32_t *>(p.out + (size_t)tok * H + f0 + f) = pack_bf16x2(v0, v1);
    }
}

// Dynamic shared memory that k_few_up may ask for, beside its static 9 KB.
constexpr int kFewUpSmem = 216 * 1024;

// Raises a kernel's dynamic shared memory limit, once per device.
template <class K>
static cudaError_t allow_smem(K kern, int bytes) {
    static LaunchMemo memo;
    int done = 0;
    return memo.get((long long)(uintptr_t)kern, &done, [&](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
}

static cudaError_t launch_few(Few p, cudaStream_t st) {
    if (p.ntok == 0) return cudaMemsetAsync(p.status, 0, 4, st);
    p.per = p.ntok < 8 ? p.ntok : 8;
    while (few_up_smem(p.H, p.per) > (size_t)kFewUpSmem) --p.per;
    const size_t up = few_up_smem(p.H, p.per);
    cudaError_t err = allow_smem(k_few_up, kFewUpSmem);
    if (err != cudaSuccess) return err;
    err = launch_kernel(k_few_up, dim3(kFewCluster, p.inter >> 7, p.ntok * p.R),
                                    dim3(kFewThreads), up, st, p);
    if (err != cudaSuccess) return err;
    const int NT = p.ntok <= 8 ? 1 : p.ntok <= 16 ? 2 : p.ntok <= 32 ? 4 : 8;
    const auto kern = NT == 1 ? k_few_down<1> : NT == 2 ? k_few_down<2> : NT == 4 ? k_few_down<4> : k_few_down<8>;
    const size_t down = few_down_smem(p.ntok, p.E, p.R, NT);
    if ((err = allow_smem(kern, 64 * 1024)) != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(p.H >> 4);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = down;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace moe

extern "C" int moe_layer_few(const moe_shape *sh, int inter, const uint16_t *x,
                             const int32_t *topk_idx, const float *topk_w, const uint8_t *w13_q,
                             const float *w13_s, const uint8_t *w2_q, const float *w2_s,
                             uint8_t *h_q, float *h_s, uint16_t *out, int32_t *status,
                             void *stream) {
    MOE_TRACE_CALL();
    moe_sizes z;
    int rc = moe_sizes_query(sh, &z);
    if (rc != MOE_OK || (rc = moe::check_width(inter)) != MOE_OK) return rc;
    const int64_t ntok = (int64_t)sh->N * sh->T, A = ntok * sh->R;
    if (ntok > MOE_FEW_MAX_TOKENS) return MOE_ENOTSUP;
    if (!moe::ok_buffer(x, z.bytes_x) || !moe::ok_buffer(topk_idx, z.bytes_topk_idx) ||
        !moe::ok_buffer(topk_w, z.bytes_topk_idx) || !moe::ok_buffer(w13_q, 1) ||
        !moe::ok_buffer(w13_s, 4) || !moe::ok_buffer(w2_q, 1) || !moe::ok_buffer(w2_s, 4) ||
        !moe::ok_buffer(h_q, A * inter) || !moe::ok_buffer(h_s, A * (inter / 128) * 4) ||
        !moe::ok_buffer(out, z.bytes_x) || !moe::ok_buffer(status, 4))
        return MOE_EINVAL;
    const moe::Few p{(int)ntok, sh->E, sh->R, sh->H, inter, 0,   x,   topk_idx, topk_w,
                     w13_q,     w13_s, w2_q,  w2_s,  h_q,   h_s, out, status};
    return moe::launch_few(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                   : MOE_ECUDA;
}
