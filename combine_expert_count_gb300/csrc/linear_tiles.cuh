// linear_tiles.cuh -- the products of 16-bit rows and weights for many rows: the kernel
// and its launch, of linear_tiles.cu (rows of outputs that start on 16 bytes) and
// linear_ragged.cu (others).
//
// Two CTAs of a cluster, on two SMs, share a tile of 256 rows by up to 256 outputs
// (or half as many of the gate and of the up projection): each brings its 128 rows of
// x and half of the tile's weights by TMA, and one issues products that both SMs'
// tensor cores work on, each with its rows against all of the weights.  A CTA alone on
// a 128 x 256 tile would fill and read 1.5 times the shared memory for the same work.
// Pairs go through the tiles one after another; an accumulator in tensor memory is
// stored by eight warps while the other one is filled.
//
// Measured: 8191 x 7168 x 7168 483 to 504 us (1.67 to 1.74 PFLOP/s, the tensor pipe is busy 83%
// of the time), gate and up of 2048 by 7168 for 8191 rows 278 (1.73), 509 x 7168 x 7168 40.9.
// What is left of the large ones is power (the clock falls) and the last round's tiles.  The
// small ones wait for what the SMs take in: 509 rows go as tiles 224 wide to 64 of the 76
// pairs, whose 440 MB take 30 us at 14.5 TB/s; the first loads and the outputs take 6 more, and
// about 5 are not accounted for.  A second pair that got the weights by the same copies went no
// faster (39.8 for 39.3).  Tiles of a short k are bound by their outputs, about 12 ns a column
// of a tile: 4346 x 3960 x 192 21 us, 24.5 where rows start on 8 bytes, 29 on 4 and 41 on 2.  k
// shared by two pairs was no faster than the clusters of the kernel for few rows.
#pragma once

#include "act.cuh"
#include "bf16.cuh"
#include "launch.h"
#include "linear.h"
#include "tc.cuh"
#include "tilemap.h"

namespace moe {

constexpr int kPairRows = 256;               // of a tile, half of them each CTA's
constexpr int kOpBytes = 128 * 128;          // 128 rows of a block along k
constexpr int kPairStages = 5, kPairStageBytes = 2 * kOpBytes;
constexpr int kOutWarps = 8, kPairTma = 8, kPairMma = 9, kPairWarps = 10;
constexpr int kPairThreads = 32 * kPairWarps;
constexpr int kOutStage = 32 * 128;          // a storing warp's staging
constexpr int kResStage = 2 * 32 * 64;       // and its residual's, two chunks
constexpr int kF32Run = 8;                   // blocks of k between the sums of an fp32 result
constexpr int kF32Width = 128;               // of its tiles at most: the sums stay in registers

struct alignas(16) PairShared {
    uint64_t full[kPairStages], empty[kPairStages], tfull[2], tempty[2], drain;
    uint32_t tmem;
    int stop;  // this CTA gave up
};
constexpr size_t kPairSmem =
    1024 + (size_t)kPairStages * kPairStageBytes + kOutWarps * (kOutStage + kResStage) + sizeof(PairShared);
static_assert(kPairSmem <= 232448, "a CTA's shared memory");

// Row tiles whose columns are gone through together, so that the pairs at work at one
// time share rows and weights in L2.
constexpr int kPairRun = 8;

struct PairTile {
    int row0, c0;  // first row of the pair, first output
};

__device__ __forceinline__ PairTile pair_tile(const Linear &p, int width, int tiles_m, int tiles_n,
                                              int t) {
    const int per = kPairRun * tiles_n, run = t / per, v = t - run * per;
    const int high = min(kPairRun, tiles_m - run * kPairRun);
    const int ni = v / high, mi = run * kPairRun + v - ni * high;
    return {mi * kPairRows, ni * width};
}

// A storing warp's 32 rows of sums lie in shared memory, 128 bytes of each at a time:
// 32 outputs, or 16 of the gate and the same 16 of the up projection.  Vector j of 16
// bytes of row r is where the lanes of a row, and of a column of rows, meet no bank
// twice.
__host__ __device__ constexpr int chunk_outs(bool pair) { return pair ? 16 : 32; }
__device__ __forceinline__ uint8_t *staged(uint8_t *stage, int r, int j) {
    return stage + r * 128 + ((j ^ r) & 7) * 16;
}

// What the outputs of a chunk take beside their sums, eight outputs of a row a lane,
// asked for before the sums are there: the bias to registers, the residual to shared
// memory (each lane reads what it copied itself).
template <bool kPair, bool kWide>
struct Beside {
    uint4 bias[kPair ? 2 : 1];
    uint8_t *res;  // two chunks' 32 rows of 64 bytes

    __device__ __forceinline__ uint4 *at_res(int r, int j, int chunk) const {
        return reinterpret_cast<uint4 *>(res + (chunk & 1) * 2048 + r * 64 + ((j ^ (r >> 1)) & 3) * 16);
    }
    __device__ __forceinline__ void load(const Linear &p, size_t row0, int rows, int c, int end,
                                         int chunk) {
        constexpr int kLanes = chunk_outs(kPair) / 8;  // of a row
        if (!kWide) return;
        const int lane = threadIdx.x & 31, at = c + (lane % kLanes) * 8;
        const bool in = at < min(end, p.n);
        if (in && p.bias) {
            bias[0] = *reinterpret_cast<const uint4 *>(p.bias + at);
            if (kPair) bias[kPair ? 1 : 0] = *reinterpret_cast<const uint4 *>(p.bias + p.n + at);
        }
        if (!kPair && p.res) {
            if (in)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 8 + lane / kLanes;
                    if (r < rows)
                        copy16_async(at_res(r, lane % kLanes, chunk), p.res + (row0 + r) * p.n + at);
                }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
};

template <int i>
struct Number {
    static constexpr int value = i;
};

// V neighbouring values as the outputs' type takes them.
template <int V>
struct Bits {
    using type = uint16_t;
};
template <>
struct Bits<2> {
    using type = uint32_t;
};
template <>
struct Bits<4> {
    using type = uint2;
};
template <int V>
__device__ __forceinline__ typename Bits<V>::type bits_at(const uint16_t *from) {
    return *reinterpret_cast<const typename Bits<V>::type *>(from);
}
__device__ __forceinline__ void widen(float (&v)[1], uint16_t w) { v[0] = bf16_lo(w); }
__device__ __forceinline__ void widen(float (&v)[2], uint32_t w) {
    v[0] = bf16_lo(w), v[1] = bf16_hi(w);
}
__device__ __forceinline__ void widen(float (&v)[4], uint2 w) {
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
}

// As finish, for any number of outputs that is a multiple of V: V of them a lane, four or
// eight rows of a lane at a time.  (One row after another a tile of 256 x 256 took 11 us.)
template <bool kPair, bool kF32, int V, bool kRes>
__device__ __forceinline__ void finish_few(const Linear &p, uint8_t *stage, size_t row0, int rows,
                                        int c, int end) {
    constexpr int kLanes = chunk_outs(kPair) / V, kRows = 32 / kLanes;  // of a row; rows at a time
    constexpr int kMost = V == 4 ? 4 : 8;  // (of kLanes times altogether)
    static_assert(kLanes % kMost == 0, "whole rounds");
    const int lane = threadIdx.x & 31, o = lane % kLanes * V, at = c + o;
    const bool in = at < end;
    float bias[V] = {}, bias2[V] = {};
    if (p.bias && in) {
        widen(bias, bits_at<V>(p.bias + at));
        if (kPair) widen(bias2, bits_at<V>(p.bias + p.n + at));
    }
    typename Bits<V>::type res[kRes ? kMost : 1] = {};
    const auto row = [&](int i) { return i * kRows + lane / kLanes; };
    const auto residual = [&](int s) {  // of a round, asked for in the one before
        if (kRes && in && s < kLanes)
#pragma unroll
            for (int i = 0; i < kMost; ++i)
                if (row(s + i) < rows)
                    res[kRes ? i : 0] = bits_at<V>(p.res + (row0 + row(s + i)) * p.n + at);
    };
    residual(0);
#pragma unroll 1
    for (int s = 0; s < kLanes && s * kRows < rows; s += kMost) {
        float a[kMost * V] = {}, b[kPair ? kMost * V : 1] = {};
        typename Bits<V>::type now[kRes ? kMost : 1];
#pragma unroll
        for (int i = 0; i < (kRes ? kMost : 1); ++i) now[i] = res[i];
        residual(s + kMost);
        const auto get = [&](float *to, int i, int from) {
            const uint8_t *place = staged(stage, row(s + i), from >> 2) + (from & 3) * 4;
            if constexpr (V == 4) {
                const float4 f = *reinterpret_cast<const float4 *>(place);
                to[0] = f.x, to[1] = f.y, to[2] = f.z, to[3] = f.w;
            } else if constexpr (V == 2) {
                const float2 f = *reinterpret_cast<const float2 *>(place);
                to[0] = f.x, to[1] = f.y;
            } else {
                to[0] = *reinterpret_cast<const float *>(place);
            }
        };
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            get(a + V * i, i, o);
            if constexpr (kPair) get(b + V * i, i, 16 + o);
        }
#pragma unroll
        for (int i = 0; i < kMost * V; ++i) a[i] += bias[i % V];
        activate<kF32>(p.act, a);
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            float *v = a + V * i, r[V];
            widen(r, now[kRes ? i : 0]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (kPair) v[e] *= b[kPair ? V * i + e : 0] + bias2[e];
                if (kRes) v[e] += r[e];
            }
            if (row(s + i) >= rows || !in) continue;
            const size_t to = (row0 + row(s + i)) * p.n + at;
            if constexpr (kF32 && V == 4)
                *reinterpret_cast<float4 *>(p.yf + to) = make_float4(v[0], v[1], v[2], v[3]);
            else if constexpr (kF32 && V == 2)
                *reinterpret_cast<float2 *>(p.yf + to) = make_float2(v[0], v[1]);
            else if constexpr (kF32)
                p.yf[to] = v[0];
            else if constexpr (V == 4)
                *reinterpret_cast<uint2 *>(p.y + to) =
                    make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            else if constexpr (V == 2)
                *reinterpret_cast<uint32_t *>(p.y + to) = pack_bf16x2(v[0], v[1]);
            else
                p.y[to] = (uint16_t)pack_bf16x2(v[0], 0.0f);
        }
    }
}

// Finishes and stores the chunk of outputs c .. of the warp's rows row0 .., rows and
// outputs (below end) as far as there are any.
template <bool kPair, bool kF32, bool kWide>
__device__ __forceinline__ void finish(const Linear &p, uint8_t *stage, const Beside<kPair, kWide> &by,
                                       size_t row0, int rows, int c, int end, int chunk) {
    constexpr int kOuts = chunk_outs(kPair), kLanes = kOuts / 8, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31;
    end = min(end, p.n);
    if (kWide) {
        // eight outputs of each of kLanes rows a lane: the lanes of a row write it together
        const int j = lane % kLanes, at = c + j * 8;
        float a[kLanes * 8] = {};
        const auto get = [&](float *to, int i, int from) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 f =
                    *reinterpret_cast<float4 *>(staged(stage, i * kRows + lane / kLanes, from + h));
                to[4 * h] = f.x, to[4 * h + 1] = f.y, to[4 * h + 2] = f.z, to[4 * h + 3] = f.w;
            }
        };
        float w[8] = {};
        if (p.bias) unpack8(w, by.bias[0]);
#pragma unroll
        for (int i = 0; i < kLanes; ++i) {
            get(a + 8 * i, i, 2 * j);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[8 * i + e] += w[e];
        }
        activate<kF32>(p.act, a);
        if (kPair && p.bias) unpack8(w, by.bias[kPair ? 1 : 0]);
        // all but the next chunk's residual is here
        if (!kPair && p.res) asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
        for (int i = 0; i < kLanes; ++i) {
            const int r = i * kRows + lane / kLanes;
            float *v = a + 8 * i;
            if (kPair) {
                float b[8] = {};
                get(b, i, 4 + 2 * j);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= b[e] + w[e];
            } else if (p.res) {
                float b[8];
                unpack8(b, *by.at_res(r, j, chunk));
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += b[e];
            }
            if (r >= rows || at >= end) continue;
            const size_t to = (row0 + r) * p.n + at;
            if (kF32) {
                *reinterpret_cast<float4 *>(p.yf + to) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4 *>(p.yf + to + 4) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                *reinterpret_cast<uint4 *>(p.y + to) =
                    make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            }
        }
        return;
    }
    // rows that do not all start on 16 bytes
    const auto few = [&](auto V) {
        if (!kPair && p.res)
            finish_few<kPair, kF32, V.value, !kPair>(p, stage, row0, rows, c, end);
        else
            finish_few<kPair, kF32, V.value, false>(p, stage, row0, rows, c, end);
    };
    if ((p.n & 3) == 0)
        few(Number<4>{});
    else if ((p.n & 1) == 0)
        few(Number<2>{});
    else
        few(Number<1>{});
}

// width: weight rows of a tile (both halves together), a multiple of 32, or of 64 for
// kPair.
template <bool kPair, bool kF32, bool kWide>
__global__ void __launch_bounds__(kPairThreads, 1)
    k_linear_tiles(const __grid_constant__ Linear p, int width, int tiles_m, int tiles_n,
                   const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ CUtensorMap map_w) {
    constexpr int kOuts = chunk_outs(kPair);
    constexpr int kAcc = kF32 ? kF32Width / 2 : 1;  // fp32 results: a thread's sums
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + align1024(smem_raw);
    uint8_t *staging = ring + kPairStages * kPairStageBytes;
    PairShared &s =
        *reinterpret_cast<PairShared *>(staging + kOutWarps * (kOutStage + kResStage));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x & 1, pairs = gridDim.x >> 1;
    const int tiles = tiles_m * tiles_n, outs = kPair ? width >> 1 : width;
    const int Kb = (p.k + kLinearBlock - 1) / kLinearBlock;

    if (tid == 0) {
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 2 * kOutWarps);
        }
        mbar_init(&s.drain, 1);
        s.stop = 0;
        fence_mbar_init();
        tma_prefetch_map(&map_x);
        tma_prefetch_map(&map_w);
    }
    if (warp == kPairMma) tc_alloc_pair<512>(&s.tmem);
    tc_fence_before();
    __syncthreads();
    // (not before the tensor memory is this CTA's: the next kernel's may take the rest)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cluster_sync();  // the other CTAs' barriers are there too
    tc_fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = s.tmem;
    volatile int *stop = &s.stop;
    int issued = 0;
    float acc[kAcc];  // fp32 results: the sums of a thread's row and half of the outputs

    if (warp == kPairTma) {
        const uint32_t one = elect_one();
        const int half = width >> 1;  // weight rows that this CTA brings
        const uint32_t bytes = 2 * (kOpBytes + half * 128);
        bool ok = true;
        for (int t = blockIdx.x >> 1; ok && t < tiles; t += pairs) {
            const PairTile tile = pair_tile(p, outs, tiles_m, tiles_n, t);
            const int xrow = tile.row0 + rank * 128;
            const int wrow = kPair ? rank * p.n + tile.c0 : tile.c0 + rank * half;
#pragma unroll 1
            for (int b = 0; b < Kb; ++b, ++issued) {
                const int st = issued % kPairStages;
                if (issued >= kPairStages &&
                    !(ok = wait_or_stop(&s.empty[st], (issued / kPairStages - 1) & 1, stop)))
                    break;
                if (!one) continue;
                uint8_t *x = ring + st * kPairStageBytes;
                const uint32_t bar = dsmem_addr(&s.full[st], 0);
                if (rank == 0) mbar_arrive_expect_tx(&s.full[st], bytes);
                tma_tile_pair(x, &map_x, b * 128, xrow, bar);
                tma_tile_pair(x + kOpBytes, &map_w, b * 128, wrow, bar);
            }
        }
        // the other CTA's last signals are here before this one goes
        for (int i = max(0, issued - kPairStages); ok && i < issued; ++i)
            ok = wait_or_stop(&s.empty[i % kPairStages], (i / kPairStages) & 1, stop);
    } else if (warp == kPairMma) {
        if (rank == 0) {
            const uint32_t one = elect_one(), idesc = tc_bf16_f32(kPairRows, width);
            const uint16_t both = 3;
            bool ok = true;
            int it = 0, run = 0;  // blocks, and accumulators filled
            for (int t = blockIdx.x >> 1; ok && t < tiles; t += pairs) {
#pragma unroll 1
                for (int b = 0; b < Kb; ++b, ++it) {
                    const int st = it % kPairStages, ac = run & 1;
                    const bool first = kF32 ? b % kF32Run == 0 : b == 0;
                    const bool last = b == Kb - 1 || (kF32 && b % kF32Run == kF32Run - 1);
                    if (first && run >= 2 &&
                        !(ok = wait_or_stop(&s.tempty[ac], (run / 2 - 1) & 1, stop)))
                        break;
                    if (!(ok = wait_or_stop(&s.full[st], (it / kPairStages) & 1, stop))) break;
                    tc_fence_after();
                    const uint64_t x = tc_operand(ring + st * kPairStageBytes);
                    const uint64_t w = tc_operand(ring + st * kPairStageBytes + kOpBytes);
                    tc_mma_bf16x64_pair(tmem + ac * 256, x, w, idesc, !first, one);
                    tc_commit_pair(&s.empty[st], both, one);
                    if (last) {
                        tc_commit_pair(&s.tfull[ac], both, one);
                        ++run;
                    }
                }
            }
        }
    } else {
        const int quad = warp & 3, half = warp >> 2;  // lanes 32 quad ..; half of the outputs
        const int cols = outs >> 1;
        const uint32_t mine = tmem + ((uint32_t)(quad * 32) << 16) + half * cols;
        const uint32_t back[2] = {dsmem_addr(&s.tempty[0], 0), dsmem_addr(&s.tempty[1], 0)};
        uint8_t *stage = staging + warp * kOutStage;
        uint8_t *residual = staging + kOutWarps * kOutStage + warp * kResStage;
        bool ok = true;
        int run = 0;
#pragma unroll 1
        for (int t = blockIdx.x >> 1; ok && t < tiles; t += pairs) {
            const PairTile tile = pair_tile(p, outs, tiles_m, tiles_n, t);
            const size_t row0 = (size_t)tile.row0 + rank * 128 + quad * 32;
            const int rows = (int)min((long long)32, (long long)p.rows - (long long)row0);
            const int c0 = tile.c0 + half * cols, end = c0 + cols;
            Beside<kPair, kWide> by = {};
            by.res = residual;
            by.load(p, row0, rows, c0, end, 0);
            if constexpr (kF32) {
#pragma unroll
                for (int i = 0; i < kAcc; ++i) acc[i] = 0.0f;
                for (int b = 0; b < Kb; b += kF32Run, ++run) {
                    const int ac = run & 1;
                    ok = __all_sync(kFull, wait_or_stop(&s.tfull[ac], (run / 2) & 1, stop));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < kAcc; j += 16) {
                        if (j >= cols) break;
                        uint32_t v[16];
                        tc_ld16(v, mine + ac * 256 + j);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[j + i] += __uint_as_float(v[i]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_at(back[ac]);
                }
            } else {
                ok = __all_sync(kFull, wait_or_stop(&s.tfull[run & 1], (run / 2) & 1, stop));
                tc_fence_after();
            }
            if (!ok) break;
            const auto chunk = [&](int c) {
                // where an accumulator ends within the 32, what is behind it is not stored
                uint32_t v[2][16];
                if constexpr (!kF32) {
                    const uint32_t ac = mine + (run & 1) * 256 + c;
                    tc_ld16(v[0], ac);
                    tc_ld16(v[1], ac + (kPair ? outs : 16));
                    tc_wait_ld();
                    if (c + kOuts >= cols) {  // all of it is in registers
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_at(back[run & 1]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i >> 4][i & 15] = __float_as_uint(acc[(c + i) % kAcc]);
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4 *>(staged(stage, lane, j)) =
                        make_uint4(v[j / 4][4 * j % 16], v[j / 4][4 * j % 16 + 1],
                                   v[j / 4][4 * j % 16 + 2], v[j / 4][4 * j % 16 + 3]);
                __syncwarp();
                const Beside<kPair, kWide> now = by;
                by.load(p, row0, rows, c0 + c + kOuts, end, c / kOuts + 1);
                finish<kPair, kF32, kWide>(p, stage, now, row0, rows, c0 + c, end, c / kOuts);
            };
            if constexpr (kF32) {
#pragma unroll
                for (int c = 0; c < kAcc; c += 32)
                    if (c < cols) chunk(c);
            } else {
#pragma unroll 1
                for (int c = 0; c < cols; c += kOuts) chunk(c);
                ++run;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (s.stop) {  // a kernel that gave up leaves no copy and no product in flight
        if (rank == 0 && warp == kPairTma && lane == 0)
            // (where the other CTA brought nothing this CTA's copies are there all the same
            // after the first of these waits)
            for (int i = max(0, issued - kPairStages); i < issued; ++i)
                if (!mbar_wait(&s.full[i % kPairStages], (i / kPairStages) & 1)) break;
        if (rank == 0 && warp == kPairMma) {
            tc_commit_one_of_pair(&s.drain, elect_one());
            mbar_wait(&s.drain, 0);
        }
        if (tid == 0 && p.status) flag(p.status, MOE_ST_TIMEOUT);
        __syncthreads();
    }
    cluster_sync();  // neither CTA goes while the other may read or signal it
    tc_fence_after();
    if (warp == kPairMma) tc_free_pair<512>(tmem);
}

template <bool kPair, bool kF32, bool kWide>
static cudaError_t launch_tiles(const Linear &p, const LinearPlan &plan, cudaStream_t st) {
    const auto kern = k_linear_tiles<kPair, kF32, kWide>;
    const int width = plan.width;
    CUtensorMap map_x, map_w;
    cudaError_t err = tile_map(&map_x, p.x, p.rows, 2 * p.k, 128);
    if (err == cudaSuccess)
        err = tile_map(&map_w, p.w, (int64_t)(kPair ? 2 : 1) * p.n, 2 * p.k, width / 2);
    if (err != cudaSuccess) return err;
    static LaunchMemo memo;
    int done = 0;
    err = memo.get(0, &done, [&](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kPairSmem);
    });
    if (err != cudaSuccess) return err;
    const int outs = kPair ? width / 2 : width;
    const int tiles_m = (p.rows + kPairRows - 1) / kPairRows, tiles_n = (p.n + outs - 1) / outs;
    const long long tiles = (long long)tiles_m * tiles_n;
    if (tiles >= 1LL << 30) return cudaErrorInvalidValue;
    const int pairs = sm_count() / 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = kPairSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p, width, tiles_m, tiles_n, map_x, map_w);
}

template <bool kWide>
static cudaError_t launch_all(const Linear &p, bool pair, const LinearPlan &plan, cudaStream_t st) {
    return pair   ? launch_tiles<true, false, kWide>(p, plan, st)
           : p.yf ? launch_tiles<false, true, kWide>(p, plan, st)
                  : launch_tiles<false, false, kWide>(p, plan, st);
}

}  // namespace moe
