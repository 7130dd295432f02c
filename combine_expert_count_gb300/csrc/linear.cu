// linear.cu -- moe_linear and moe_linear_glu: products of bf16 rows and weights with
// their epilogue.
#include <cooperative_groups.h>

#include "act.cuh"
#include "bf16.cuh"
#include "check.h"
#include "launch.h"
#include "linear.h"
#include "tc.cuh"
#include "tilemap.h"
#include "trace.h"

namespace moe {

namespace cg = cooperative_groups;

// The weights are the 128-row operand of the tensor cores and NR rows of x the other:
// a lane of tensor memory is an output.  A CTA has 128 outputs (of both halves) of NR
// rows; a warp brings blocks of 64 along k by TMA into a ring, one issues their
// products, four take the sums out.  The CTAs of a cluster share k and then the rows:
// each adds up and stores its own of them.
constexpr int kLinTma = 4, kLinMma = 5, kLinWarps = 6, kLinThreads = 32 * kLinWarps;
constexpr int kLinTile = 128 * 128;  // bytes of a weight tile of a stage
#ifndef F32RUN
#define F32RUN 8
#endif
constexpr int kLinRun = F32RUN;           // blocks of k between the sums of an fp32 result

__host__ __device__ constexpr int lin_stage(int NR, bool pair) {
    return (pair ? 2 : 1) * kLinTile + NR * 128;
}
// two CTAs an SM up to 64 rows
__host__ __device__ constexpr int lin_stages(int NR, bool pair) {
    return (NR <= 64 ? 111 * 1024 : 220 * 1024) / lin_stage(NR, pair);
}
template <int kStages>
struct alignas(16) LinShared {
    uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], drain;
    uint32_t tmem;
    int stop;
};
template <int NR, bool kPair>
constexpr size_t lin_smem() {
    return 1024 + (size_t)lin_stages(NR, kPair) * lin_stage(NR, kPair) +
           sizeof(LinShared<lin_stages(NR, kPair)>);
}

// The outputs of a CTA's rows from their sums, which lie in shared memory as
// [half][row][128 outputs] of each part: added in the parts' order.  A lane has eight
// outputs of kAtOnce rows, 16 lanes a row.
constexpr int kAtOnce = 4;

template <int NR, bool kPair, bool kF32>
struct Finish {
    const Linear &p;
    uint32_t sums;  // shared-memory address
    int parts, row0, m, c0;

    __device__ __forceinline__ uint32_t at(int q, int h, int j, int o) const {
        uint32_t a;
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(a)
            : "r"(sums + ((h * NR + j) * 128 + o) * 4), "r"(q));
        return a;
    }

    // n is a multiple of 8; rows j, j + step, ...
    __device__ __forceinline__ void vectors(int j, int step, const uint4 (&bias)[2],
                                            const uint4 (&res)[kAtOnce]) const {
        const int o = (threadIdx.x & 15) * 8, c = c0 + o;
        float a[8 * kAtOnce] = {}, b[kPair ? 8 * kAtOnce : 8] = {};
#pragma unroll 1
        for (int q = 0; q < parts; ++q)
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int r = min(j + i * step, m - 1);
#pragma unroll
                for (int h = 0; h < (kPair ? 4 : 2); ++h) {
                    const float4 f = ld_dsmem4(at(q, h >> 1, r, o + (h & 1) * 4));
                    float *to = (h >> 1 ? b : a) + 8 * i + (h & 1) * 4;
                    to[0] += f.x, to[1] += f.y, to[2] += f.z, to[3] += f.w;
                }
            }
        float w[8];
        if (p.bias) {
            unpack8(w, bias[0]);
#pragma unroll
            for (int i = 0; i < 8 * kAtOnce; ++i) a[i] += w[i & 7];
        }
        activate<kF32>(p.act, a);
        if (kPair) {
            if (p.bias) {
                unpack8(w, bias[1]);
#pragma unroll
                for (int i = 0; i < 8 * kAtOnce; ++i) b[kPair ? i : 0] += w[i & 7];
            }
#pragma unroll
            for (int i = 0; i < 8 * kAtOnce; ++i) a[i] *= b[kPair ? i : 0];
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int r = j + i * step;
            if (r >= m || c >= p.n) continue;
            float *v = a + 8 * i;
            if (!kPair && p.res) {
                unpack8(w, res[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += w[e];
            }
            const size_t to = (size_t)(row0 + r) * p.n + c;
            if (kF32) {
                *reinterpret_cast<float4 *>(p.yf + to) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4 *>(p.yf + to + 4) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                *reinterpret_cast<uint4 *>(p.y + to) =
                    make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            }
        }
    }

    // any n: one output of row j a lane at a time
    __device__ __forceinline__ void scalars(int j) const {
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        for (int o = lane; o < 128 && c0 + o < p.n; o += 32) {
            const int c = c0 + o;
            float a[1] = {0.0f}, b = 0.0f;
            for (int q = 0; q < parts; ++q) {
                a[0] += ld_dsmemf(at(q, 0, j, o));
                if (kPair) b += ld_dsmemf(at(q, 1, j, o));
            }
            if (p.bias) {
                a[0] += bf16_lo(__ldg(p.bias + c));
                if (kPair) b += bf16_lo(__ldg(p.bias + p.n + c));
            }
            activate<kF32>(p.act, a);
            if (kPair) a[0] *= b;
            const size_t to = (size_t)(row0 + j) * p.n + c;
            if (!kPair && p.res) a[0] += bf16_lo(p.res[to]);
            if (kF32)
                p.yf[to] = a[0];
            else
                p.y[to] = (uint16_t)pack_bf16x2(a[0], 0.0f);
        }
    }
};

template <int NR, bool kPair, bool kF32>
__global__ void __launch_bounds__(kLinThreads, NR <= 64 ? 2 : 1)
    k_linear(const __grid_constant__ Linear p, const __grid_constant__ CUtensorMap map_x,
             const __grid_constant__ CUtensorMap map_w) {
    constexpr int kStages = lin_stages(NR, kPair), kBytes = lin_stage(NR, kPair);
    constexpr int kHalves = kPair ? 2 : 1;
    constexpr int kAccs = kF32 ? 2 : 1;  // accumulators
    constexpr int kUsed = kAccs * kHalves * NR, kCols = kUsed < 32 ? 32 : kUsed;
    static_assert(kHalves * NR * 512 <= kStages * kBytes, "the sums go through the ring");
    using Shared = LinShared<kStages>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + align1024(smem_raw);
    Shared &s = *reinterpret_cast<Shared *>(ring + kStages * kBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c0 = blockIdx.y * 128, row0 = blockIdx.x * NR, m = min(NR, p.rows - row0);
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = (int)gridDim.z, part = (int)blockIdx.z;
    const int Kb = (p.k + kLinearBlock - 1) / kLinearBlock;
    const int b0 = (int)((long long)Kb * part / parts), b1 = (int)((long long)Kb * (part + 1) / parts);

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 4);
        }
        mbar_init(&s.drain, 1);
        s.stop = 0;
        fence_mbar_init();
        tma_prefetch_map(&map_x);
        tma_prefetch_map(&map_w);
    }
    if (warp == kLinMma) tc_alloc<kCols>(&s.tmem);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile int *stop = &s.stop;
    float *left = reinterpret_cast<float *>(ring);  // [half][row][128], once the ring is done
    int issued = 0;  // blocks whose loads are under way (TMA warp)

    if (warp == kLinTma) {
        const uint32_t one = elect_one();
        for (int b = b0; b < b1; ++b, ++issued) {
            const int st = issued % kStages;
            if (issued >= kStages && !wait_or_stop(&s.empty[st], (issued / kStages - 1) & 1, stop))
                break;
            if (!one) continue;
            uint8_t *w = ring + st * kBytes;
            mbar_arrive_expect_tx(&s.full[st], kBytes);
            tma_tile(w, &map_w, b * 128, c0, &s.full[st]);
            if (kPair) tma_tile(w + kLinTile, &map_w, b * 128, p.n + c0, &s.full[st]);
            tma_tile(w + kHalves * kLinTile, &map_x, b * 128, row0, &s.full[st]);
        }
    } else if (warp == kLinMma) {
        const uint32_t one = elect_one(), idesc = tc_bf16_f32(128, NR);
        for (int it = 0; it < b1 - b0; ++it) {
            const int st = it % kStages;
            const int run = kF32 ? it / kLinRun : 0, ac = run & 1;
            const bool first = kF32 ? it % kLinRun == 0 : it == 0;
            const bool last = it == b1 - b0 - 1 || (kF32 && it % kLinRun == kLinRun - 1);
            if (first && run >= 2 && !wait_or_stop(&s.tempty[ac], (run / 2 - 1) & 1, stop)) break;
            if (!wait_or_stop(&s.full[st], (it / kStages) & 1, stop)) break;
            tc_fence_after();
            const uint64_t w = tc_operand(ring + st * kBytes);
            const uint64_t x = tc_operand(ring + st * kBytes + kHalves * kLinTile);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 bytes along k: 2 address units
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    tc_mma_bf16(tmem + (ac * kHalves + h) * NR, w + h * (kLinTile >> 4) + kk * 2,
                                x + kk * 2, idesc, !first || kk > 0, one);
            tc_commit(&s.empty[st], one);
            if (last) tc_commit(&s.tfull[ac], one);
        }
    } else {
        const uint32_t mine = tmem + ((uint32_t)(warp * 32) << 16);
        if constexpr (kF32) {
            float acc[NR] = {};
            const int runs = (b1 - b0 + kLinRun - 1) / kLinRun;
            bool ok = true;
            for (int run = 0; ok && run < runs; ++run) {
                const int ac = run & 1;
                ok = __all_sync(kFull, wait_or_stop(&s.tfull[ac], (run / 2) & 1, stop));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < NR; j += 16) {
                    uint32_t v[16];
                    tc_ld16(v, mine + ac * NR + j);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[j + i] += __uint_as_float(v[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.tempty[ac]);
            }
            // the last products are done: the ring is free
#pragma unroll
            for (int j = 0; j < NR; ++j)
                if (j < m) left[j * 128 + tid] = acc[j];
        } else if (__all_sync(kFull, wait_or_stop(&s.tfull[0], 0, stop))) {
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < kHalves * NR; j += 16) {
                uint32_t v[16];
                tc_ld16(v, mine + j);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) left[(j + i) * 128 + tid] = __uint_as_float(v[i]);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (s.stop) {  // a kernel that gave up leaves no copy and no product in flight
        if (warp == kLinTma && lane == 0)
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait(&s.full[i % kStages], (i / kStages) & 1);
        if (warp == kLinMma) {
            tc_commit(&s.drain, elect_one());
            mbar_wait(&s.drain, 0);
        }
        if (tid == 0 && p.status) flag(p.status, MOE_ST_TIMEOUT);
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kLinMma) tc_free<kCols>(tmem);
    // what the outputs take beside their sums, asked for before those are there
    const int step = 2 * parts * kLinWarps, c = c0 + (lane & 15) * 8;
    int j = (part * kLinWarps + warp) * 2 + (lane >> 4);
    const bool whole = (p.n & 7) == 0, in = whole && c < p.n;
    uint4 bias[2] = {}, res[kAtOnce] = {};
    if (in && p.bias) {
        bias[0] = __ldg(reinterpret_cast<const uint4 *>(p.bias + c));
        if (kPair) bias[1] = __ldg(reinterpret_cast<const uint4 *>(p.bias + p.n + c));
    }
    const auto residual = [&]() {
        if (!kPair && in && p.res)
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (j + i * step < m)
                    res[i] = *reinterpret_cast<const uint4 *>(
                        p.res + (size_t)(row0 + j + i * step) * p.n + c);
    };
    residual();
    // where a part gave up the sums are not whole and no part stores any
    if (parts > 1) cluster.sync();
    const int any = ld_dsmem(dsmem_addr(&s.stop, min(lane, parts - 1)));
    if (!__any_sync(kFull, any)) {
        const Finish<NR, kPair, kF32> f = {p, smem_addr(left), parts, row0, m, c0};
        if (whole) {
#pragma unroll 1
            for (; j < m; j += kAtOnce * step) {
                f.vectors(j, step, bias, res);
                if (j + kAtOnce * step < m) {
                    j += kAtOnce * step;
                    residual();
                    j -= kAtOnce * step;
                }
            }
        } else {
            for (int r = part * kLinWarps + warp; r < m; r += parts * kLinWarps) f.scalars(r);
        }
    }
    if (parts > 1) cluster.sync();  // no part goes while it is read
}

// ------------------------------------------------------------ host

template <int NR, bool kPair, bool kF32>
static cudaError_t launch_few(const Linear &p, const LinearPlan &plan, cudaStream_t st) {
    const auto kern = k_linear<NR, kPair, kF32>;
    constexpr size_t kSmem = lin_smem<NR, kPair>();
    static_assert(kSmem <= (NR <= 64 ? 113 * 1024 : 232448), "CTAs of an SM");
    CUtensorMap map_x, map_w;
    cudaError_t err = tile_map(&map_x, p.x, p.rows, 2 * p.k, NR);
    if (err == cudaSuccess) err = tile_map(&map_w, p.w, (int64_t)(kPair ? 2 : 1) * p.n, 2 * p.k, 128);
    if (err != cudaSuccess) return err;
    static LaunchMemo memo;
    int done = 0;
    err = memo.get(0, &done, [&](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    });
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = (unsigned)plan.parts;
    cfg.gridDim = dim3((unsigned)((p.rows + NR - 1) / NR), (unsigned)((p.n + 127) / 128),
                       (unsigned)plan.parts);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p, map_x, map_w);
}

template <bool kPair, bool kF32>
static cudaError_t launch_at(const Linear &p, const LinearPlan &plan, cudaStream_t st) {
    if (plan.at == 16) return launch_few<16, kPair, kF32>(p, plan, st);
    if (plan.at == 32) return launch_few<32, kPair, kF32>(p, plan, st);
    if constexpr (kF32) {
        return launch_few<64, kPair, kF32>(p, plan, st);
    } else {
        if (plan.at == 64) return launch_few<64, kPair, kF32>(p, plan, st);
        if constexpr (kPair) {
            return launch_few<128, kPair, kF32>(p, plan, st);
        } else {
            if (plan.at == 128) return launch_few<128, kPair, kF32>(p, plan, st);
            return launch_few<256, kPair, kF32>(p, plan, st);
        }
    }
}

cudaError_t launch_linear(const Linear &p, bool pair, cudaStream_t st) {
    const LinearPlan plan = linear_plan(p.rows, p.n, p.k, pair, p.yf != nullptr, sm_count());
    if (plan.width) return launch_linear_tiles(p, pair, plan, st);
    if (pair) return launch_at<true, false>(p, plan, st);
    return p.yf ? launch_at<false, true>(p, plan, st) : launch_at<false, false>(p, plan, st);
}

// What both calls check; n counts all outputs.
static int check_linear(const moe_shape *sh, int64_t n, int k, int act, const uint16_t *x,
                        const uint16_t *w, const uint16_t *bias, int32_t *status, int64_t *rows) {
    moe_sizes z;
    const int rc = moe_sizes_query(sh, &z);
    if (rc != MOE_OK) return rc;
    if (n <= 0 || k <= 0 || k % 8 != 0 || act < MOE_ACT_NONE || act > MOE_ACT_SIGMOID)
        return MOE_EINVAL;
    if (n > MOE_LINEAR_MAX_N || k > 65536) return MOE_ENOTSUP;
    *rows = (int64_t)sh->N * sh->T;
    if (!ok_buffer(x, *rows * k * 2) || !ok_buffer(w, n * k * 2) || !ok_optional(bias) ||
        !ok_optional(status))
        return MOE_EINVAL;
    return *rows < ((int64_t)1 << 31) - 256 ? MOE_OK : MOE_ENOTSUP;
}

}  // namespace moe

extern "C" int moe_linear(const moe_shape *sh, int n, int k, int act, const uint16_t *x,
                          const uint16_t *w, const uint16_t *bias, const uint16_t *res,
                          uint16_t *y_bf16, float *y_f32, int32_t *status, void *stream) {
    MOE_TRACE_CALL();
    int64_t rows;
    const int rc = moe::check_linear(sh, n, k, act, x, w, bias, status, &rows);
    if (rc != MOE_OK) return rc;
    if (!moe::ok_optional(res) || !moe::ok_optional(y_bf16) || !moe::ok_optional(y_f32))
        return MOE_EINVAL;
    if (rows == 0) return MOE_OK;
    if ((y_bf16 == nullptr) == (y_f32 == nullptr)) return MOE_EINVAL;
    const moe::Linear p = {(int)rows, n, k, act, x, w, bias, res, y_bf16, y_f32, status};
    return moe::launch_linear(p, false, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ECUDA;
}

extern "C" int moe_linear_glu(const moe_shape *sh, int inter, int k, int act, const uint16_t *x,
                              const uint16_t *w13, const uint16_t *bias13, uint16_t *h,
                              int32_t *status, void *stream) {
    MOE_TRACE_CALL();
    int64_t rows;
    const int rc =
        moe::check_linear(sh, 2 * (int64_t)inter, k, act, x, w13, bias13, status, &rows);
    if (rc != MOE_OK) return rc;
    if (!moe::ok_buffer(h, rows * inter * 2)) return MOE_EINVAL;
    if (rows == 0) return MOE_OK;
    const moe::Linear p = {(int)rows, inter, k, act, x, w13, bias13, nullptr, h, nullptr, status};
    return moe::launch_linear(p, true, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ECUDA;
}
