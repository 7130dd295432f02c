// linear.cu -- moe_linear and moe_linear_glu: products of bf16 rows and weights with
// their epilogue.
#include "act.cuh"
#include "bf16.cuh"
#include "check.h"
#include "launch.h"
#include "linear.h"
#include "tc.cuh"
#include "tilemap.h"
#include "trace.h"

namespace moe {

// Few rows.  The weights are the 128-row operand of the tensor cores and NR rows of x
// the other: a lane of tensor memory is an output.  A CTA has 128 outputs, or 64 of the
// gate and the same 64 of the up projection, of NR rows; a warp brings pairs of blocks
// of 64 along k by TMA into a ring, one issues their products, four take the sums out, and
// two more help with the outputs.  (A stage costs the warps that load and issue about 300
// cycles, whatever it holds: with a block a stage a CTA took no more than 108 GB/s.)  The
// CTAs of a cluster share k and then the rows: each sends its sums of four rows at a
// time to the part that adds them up, in the parts' order, and stores them.
//
// What bounds it, and what it measured: one row, its weights.  1 x 7168 x 2048 takes 7.9 us
// (3.7 TB/s), gate and up of 2048 by 7168 11.8 (5.0 TB/s): about 2 us pass before the first
// bytes are here, 5 and 9 with weights on the way, and 1 with sums and outputs.  61 rows of
// gate and up of 768 by 2048 5.0 us, 100 x 7168 x 2048 10.6, 2048 x 256 x 7168 14.3 in fp32
// (13.3 in bf16): there a CTA's operands arrive for 7.6 us (120 GB/s an SM, which is what an
// SM takes in), 1.8 us go with sending 48 KB of sums across the cluster (14 bytes a clock),
// 2 with waiting for each other's and 1 with the outputs.  Word by word, instead of by
// vectors of four rows, the sums took 2.9 us, and read from the other CTAs' memory by those
// that add them up 20.  The sums of 128 rows wait until the ring is free: with room of
// their own, and a stage less, the fp32 case took 15.7.
constexpr int kLinTma = 4, kLinMma = 5, kLinWarps = 8, kLinThreads = 32 * kLinWarps;
constexpr int kLinTile = 128 * 128;  // bytes of a weight tile of a block of k
constexpr int kLinRun = 4;           // stages between the sums of an fp32 result: 512 of k
constexpr int kLinMostStages = 6;

struct LinShared {
    uint64_t full[kLinMostStages], empty[kLinMostStages], tfull[2], tempty[2], drain;
    uint32_t tmem;
    int stop, any;  // this part gave up; some part did
};
constexpr int kLinHead = 256;  // bytes: LinShared, before the ring
static_assert(sizeof(LinShared) <= kLinHead, "its place before the ring");
static_assert(kLinHead + 1024 == kFewHead && kLinTile == kFewTile, "the plan's");
// The rows of a part: whole groups of four, which go to it together.  Where there are
// more parts than groups the last parts have none.
__device__ __forceinline__ int lin_rows(int NR, int parts) {
    return NR / parts < 4 ? 4 : NR / parts;
}

template <int NR, bool kPair, bool kF32>
__global__ void __launch_bounds__(kLinThreads, 1)
    k_linear(const __grid_constant__ Linear p, int stages, const __grid_constant__ CUtensorMap map_x,
             const __grid_constant__ CUtensorMap map_w) {
    constexpr int kBytes = 2 * (kLinTile + NR * 128);  // two blocks of weights, then two of rows
    constexpr int kAccs = kF32 ? 2 : 1;                // accumulators
    constexpr int kUsed = kAccs * NR, kCols = kUsed < 32 ? 32 : kUsed;
    extern __shared__ uint8_t smem_raw[];
    LinShared &s = *reinterpret_cast<LinShared *>(smem_raw);
    uint8_t *ring = smem_raw + kLinHead + align1024(smem_raw + kLinHead);
    // sums [part][group of four rows][128][4] of the rows that are this part's
    constexpr bool kApart = NR <= kLinearApart;
    uint8_t *left = kApart ? ring + stages * kBytes : ring;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c0 = blockIdx.y * (kPair ? 64 : 128), row0 = blockIdx.x * NR;
    const int m = min(NR, p.rows - row0);
    const int parts = (int)gridDim.z, part = (int)blockIdx.z;
    const int Kb = (p.k + 2 * kLinearBlock - 1) / (2 * kLinearBlock);  // stages of k
    const int b0 = (int)((long long)Kb * part / parts), b1 = (int)((long long)Kb * (part + 1) / parts);

    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 4);
        }
        mbar_init(&s.drain, 1);
        s.stop = s.any = 0;
        fence_mbar_init();
        tma_prefetch_map(&map_x);
        tma_prefetch_map(&map_w);
    }
    if (warp == kLinMma) tc_alloc<kCols>(&s.tmem);
    tc_fence_before();
    __syncthreads();
    // (not before the tensor memory is this CTA's: the next kernel's may take the rest)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_after();
    if (parts > 1) cluster_arrive();  // this part is there: others may write to it
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = s.tmem;
    volatile int *stop = &s.stop;
    int issued = 0;  // blocks whose loads are under way (TMA warp)
    float acc[kF32 ? NR : 1] = {};

    if (warp == kLinTma) {
        const uint32_t one = elect_one();
        int st = 0, phase = 1;
        for (int b = b0; b < b1; ++b, ++issued) {
            if (issued >= stages && !wait_or_stop(&s.empty[st], phase, stop)) break;
            if (one) {
                uint8_t *w = ring + st * kBytes;
                mbar_arrive_expect_tx(&s.full[st], kBytes);
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // a block behind k's end is zeros
                    const int at = (2 * b + i) * 128;
                    tma_tile(w + i * kLinTile, &map_w, at, c0, &s.full[st]);
                    if (kPair)
                        tma_tile(w + i * kLinTile + kLinTile / 2, &map_w, at, p.n + c0, &s.full[st]);
                    tma_tile(w + 2 * kLinTile + i * NR * 128, &map_x, at, row0, &s.full[st]);
                }
            }
            if (++st == stages) st = 0, phase ^= 1;
        }
    } else if (warp == kLinMma) {
        const uint32_t one = elect_one(), idesc = tc_bf16_f32(128, NR);
        int st = 0, phase = 0;
        for (int it = 0; it < b1 - b0; ++it) {
            const int run = kF32 ? it / kLinRun : 0, ac = run & 1;
            const bool first = kF32 ? it % kLinRun == 0 : it == 0;
            const bool last = it == b1 - b0 - 1 || (kF32 && it % kLinRun == kLinRun - 1);
            if (first && run >= 2 && !wait_or_stop(&s.tempty[ac], (run / 2 - 1) & 1, stop)) break;
            if (!wait_or_stop(&s.full[st], phase, stop)) break;
            tc_fence_after();
            const uint64_t w = tc_operand(ring + st * kBytes);
            const uint64_t x = tc_operand(ring + st * kBytes + 2 * kLinTile);
            tc_mma_bf16x64(tmem + ac * NR, w, x, idesc, !first, one);
            tc_mma_bf16x64(tmem + ac * NR, w + (kLinTile >> 4), x + (NR * 128 >> 4), idesc, true, one);
            tc_commit(&s.empty[st], one);
            if (last) tc_commit(&s.tfull[ac], one);
            if (++st == stages) st = 0, phase ^= 1;
        }
    } else if (warp > kLinMma) {
        // these only help with the outputs
    } else if constexpr (kF32) {
        const uint32_t mine = tmem + ((uint32_t)(warp * 32) << 16);
        const int runs = (b1 - b0 + kLinRun - 1) / kLinRun;
        for (int run = 0; run < runs; ++run) {
            const int ac = run & 1;
            if (!__all_sync(kFull, wait_or_stop(&s.tfull[ac], (run / 2) & 1, stop))) break;
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
    } else {
        wait_or_stop(&s.tfull[0], 0, stop);
    }

    // ---------------------------------------------------------------- the sums to their rows' parts
    // A warp has 32 outputs of every kStep-th group of four rows, an output a lane; after
    // their activation two lanes exchange, so that one has two outputs of the first two
    // rows (unless their number is odd).
    constexpr int kAcross = kPair ? 2 : 4, kStep = kLinWarps / kAcross;
    constexpr int kMany = NR / (kPair ? 32 : 8), kAtOnce = kMany < 1 ? 1 : kMany > 4 ? 4 : kMany;
    const int LR = lin_rows(NR, parts), shift = __ffs(LR) - 1;  // rows of a part
    const int mm = min(m - part * LR, LR);                      // as many as there are
    const int across = warp % kAcross * 32 + lane, g0 = warp / kAcross;
    const bool even = (p.n & 1) == 0;
    const int col = c0 + (even ? across & ~1 : across), r0 = g0 * 4 + (even ? 2 * (lane & 1) : 0);
    const size_t y0 = ((size_t)row0 + part * LR + r0) * p.n + col;
    // what the outputs take beside their sums is asked for before those are there
    float bias = 0.0f, bias2 = 0.0f;
    if (p.bias && c0 + across < p.n) {
        bias = bf16_lo(p.bias[c0 + across]);
        if (kPair) bias2 = bf16_lo(p.bias[p.n + c0 + across]);
    }
    uint32_t res[kPair ? 1 : kAtOnce][2] = {};
    const auto residual = [&](int g) {  // of groups g0 + g, + kStep, ...
        if (!kPair && p.res)
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = (g + i * kStep) * 4 + (even ? h : 2 * h);
                    const uint16_t *from = p.res + y0 + (size_t)r * p.n;
                    uint32_t &to = res[kPair ? 0 : i][h];
                    if (r0 + r >= mm || col >= p.n) continue;
                    if (even) {
                        to = *reinterpret_cast<const uint32_t *>(from);
                    } else {
                        to = from[0];
                        if (r0 + r + 1 < mm) to |= (uint32_t)from[p.n] << 16;
                    }
                }
    };
    residual(0);
    tc_fence_before();
    __syncthreads();
    if (s.stop) {  // a kernel that gave up leaves no copy and no product in flight
        if (warp == kLinTma && lane == 0)
            for (int i = max(0, issued - stages); i < issued; ++i)
                mbar_wait(&s.full[i % stages], (i / stages) & 1);
        if (warp == kLinMma) {
            tc_commit(&s.drain, elect_one());
            mbar_wait(&s.drain, 0);
        }
        if (tid == 0 && p.status) flag(p.status, MOE_ST_TIMEOUT);
        __syncthreads();
    }
    tc_fence_after();
    if (parts > 1) {
        cluster_wait();
        if (!kApart) cluster_sync();  // all parts are done with their rings
        if (s.stop && tid < parts) st_dsmem(dsmem_addr(&s.any, tid), 1);
    }
    constexpr bool kAll = NR == 128 && !kF32;  // eight warps take the sums out
    if ((warp < 4 || kAll) && !s.stop) {
        const uint32_t mine = tmem + ((uint32_t)(warp & 3) * 32 << 16);
        uint8_t *const to = left + part * LR * 512 + (tid & 127) * 16;
        // rows j .. j + 3 to their part
        const auto leave = [&](int j, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
            if (j >= m) return;
            uint8_t *const at = to + (j & (LR - 1)) * 512;
            if (parts > 1)
                st_dsmem4(dsmem_addr(at, j >> shift), a, b, c, d);
            else
                *reinterpret_cast<uint4 *>(at) = make_uint4(a, b, c, d);
        };
        if constexpr (kF32) {
#pragma unroll
            for (int j = 0; j < NR; j += 4)
                leave(j, __float_as_uint(acc[kF32 ? j : 0]), __float_as_uint(acc[kF32 ? j + 1 : 0]),
                      __float_as_uint(acc[kF32 ? j + 2 : 0]), __float_as_uint(acc[kF32 ? j + 3 : 0]));
        } else {
            constexpr int kSets = NR < 32 ? 1 : 2;  // of 16 rows
#pragma unroll 1
            for (int j = (warp >> 2) * 32; j < m; j += 16 * kSets * (kAll ? 2 : 1)) {
                uint32_t v[kSets][16];
#pragma unroll
                for (int h = 0; h < kSets; ++h) tc_ld16(v[h], mine + j + 16 * h);
                tc_wait_ld();
#pragma unroll
                for (int h = 0; h < kSets; ++h)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        leave(j + 16 * h + i, v[h][i], v[h][i + 1], v[h][i + 2], v[h][i + 3]);
            }
        }
    }
    tc_fence_before();
    if (parts > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == kLinMma) tc_free<kCols>(tmem);

    // ---------------------------------------------------------------- the outputs
    // where a part gave up the sums are not whole and no part stores any
    if (s.any || s.stop) return;
    const uint8_t *sums = left + across * 16;
#pragma unroll 1
    for (int g = 0; (g0 + g) * 4 < mm; g += kAtOnce * kStep) {
        float a[kAtOnce * 4] = {}, b[kPair ? kAtOnce * 4 : 1] = {};
        int at[kAtOnce];  // (one group is taken again where there are no more)
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) at[i] = min(g0 + g + i * kStep, LR / 4 - 1) * 2048;
        const uint8_t *from = sums;
        for (int q = 0; q < parts; ++q, from += LR * 512)  // in the parts' order
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const float4 f = *reinterpret_cast<const float4 *>(from + at[i]);
                a[i * 4] += f.x, a[i * 4 + 1] += f.y, a[i * 4 + 2] += f.z, a[i * 4 + 3] += f.w;
                if constexpr (kPair) {
                    const float4 e = *reinterpret_cast<const float4 *>(from + at[i] + 64 * 16);
                    b[i * 4] += e.x, b[i * 4 + 1] += e.y, b[i * 4 + 2] += e.z, b[i * 4 + 3] += e.w;
                }
            }
#pragma unroll
        for (int i = 0; i < kAtOnce * 4; ++i) a[i] += bias;
        activate<kF32>(p.act, a);
        if (kPair)
#pragma unroll
            for (int i = 0; i < kAtOnce * 4; ++i) a[i] *= b[kPair ? i : 0] + bias2;
        const bool odd = lane & 1;
        float v[kAtOnce][2][2];  // of two rows two outputs, or of four rows one
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (even) {
                    const float other =
                        __shfl_xor_sync(kFull, odd ? a[4 * i + h] : a[4 * i + 2 + h], 1);
                    v[i][h][0] = odd ? other : a[4 * i + h];
                    v[i][h][1] = odd ? a[4 * i + 2 + h] : other;
                } else {
                    v[i][h][0] = a[4 * i + 2 * h];
                    v[i][h][1] = a[4 * i + 2 * h + 1];
                }
                if (!kPair) {
                    v[i][h][0] += bf16_lo(res[kPair ? 0 : i][h]);
                    v[i][h][1] += bf16_hi(res[kPair ? 0 : i][h]);
                }
            }
        if (col < p.n && even) {
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = (g + i * kStep) * 4 + h;
                    const size_t to = y0 + (size_t)r * p.n;
                    if (r0 + r >= mm) continue;
                    if (kF32)
                        *reinterpret_cast<float2 *>(p.yf + to) = make_float2(v[i][h][0], v[i][h][1]);
                    else
                        *reinterpret_cast<uint32_t *>(p.y + to) =
                            pack_bf16x2(v[i][h][0], v[i][h][1]);
                }
        } else if (col < p.n) {
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int r = (g + i * kStep) * 4 + h;
                    const size_t to = y0 + (size_t)r * p.n;
                    if (r0 + r >= mm) continue;
                    if (kF32)
                        p.yf[to] = v[i][h / 2][h % 2];
                    else
                        p.y[to] = (uint16_t)pack_bf16x2(v[i][h / 2][h % 2], 0.0f);
                }
        }
        residual(g + kAtOnce * kStep);
    }
}

// ------------------------------------------------------------ host

template <int NR, bool kPair, bool kF32>
static cudaError_t launch_few(const Linear &p, const LinearPlan &plan, cudaStream_t st) {
    const auto kern = k_linear<NR, kPair, kF32>;
    static_assert(few_stage(NR) == 2 * (kLinTile + NR * 128), "the kernel's");
    CUtensorMap map_x, map_w;
    cudaError_t err = tile_map(&map_x, p.x, p.rows, 2 * p.k, NR);
    if (err == cudaSuccess)
        err = tile_map(&map_w, p.w, (int64_t)(kPair ? 2 : 1) * p.n, 2 * p.k, kPair ? 64 : 128);
    if (err != cudaSuccess) return err;
    static LaunchMemo memo;
    int done = 0;
    err = memo.get(0, &done, [&](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
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
    const int outs = kPair ? 64 : 128;
    cfg.gridDim = dim3((unsigned)((p.rows + NR - 1) / NR), (unsigned)((p.n + outs - 1) / outs),
                       (unsigned)plan.parts);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = (size_t)(few_fixed(NR, plan.parts) + plan.stages * few_stage(NR));
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p, plan.stages, map_x, map_w);
}

template <bool kPair, bool kF32>
static cudaError_t launch_at(const Linear &p, const LinearPlan &plan, cudaStream_t st) {
    if (plan.at == 16) return launch_few<16, kPair, kF32>(p, plan, st);
    if (plan.at == 32) return launch_few<32, kPair, kF32>(p, plan, st);
    if (plan.at == 64) return launch_few<64, kPair, kF32>(p, plan, st);
    return launch_few<128, kPair, kF32>(p, plan, st);
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
