// experts.cu -- the experts' products over the grouped rows: moe_expert_gemm
// and moe_expert_gemm_swiglu.
//
// p[i][c] = sum over blocks b of 128 along k of
//           (a_s[i][b] * w_s[e][c/128][b]) * sum_{kk in b} a_q[i][kk] * w_q[e][c][kk]
//
// One persistent CTA per SM works through tiles of 128 rows of one expert by
// two column blocks of 128 (two neighbours of the plain product; the gate
// block and the up block of the same activations of the other).  One warp
// loads the operands' 128-byte-wide k blocks by TMA into a ring of four
// stages; one issues the tcgen05 products of a block into one of two
// 256-column accumulators in tensor memory; eight warps take each finished
// block out of there and add it, times its two scales, to fp32 sums that stay
// in registers over the whole of k; two bring the scales.  The fp32 scales of
// a block are why the sums leave tensor memory at every block: the tensor cores
// can only apply power-of-two scales by themselves.  A thread holds one row, so
// its row's scale is one number for all its columns, and the gate, the up value
// and half of the block maximum of an activation meet in one thread.
//
// What bounds it.  A decode batch: HBM, each weight being read once (32 experts of
// 7168 x 2048 with 64 rows each 81 us, 6.2 TB/s; gate/up of 2048 by 7168 157 us, 6.1
// TB/s).  Many rows: the sums.  8191 x 7168 x 7168 takes 308 to 330 us alone (2.55 to
// 2.73 PFLOP/s, a bf16 product's measured rate being 1.89) and 354 to 365 under
// sustained load, the uneven prefill gate/up 760 to 833 us and 850 to 870.  That is
// about 880 cycles a k block (12 rounds of 56 blocks on an SM), of which the products
// are 512.  By clock readings around the waits, which make it 1030, the sum warps
// wait 176 for products, take 486 to read an accumulator and give it back, and need
// the other 370 for scales, the last multiply-adds and, once a tile, the output; the
// warp that issues waits 424 for an accumulator.  (128 x 256 fused multiply-adds are
// 256 cycles of an SM's fp32 lanes; the loop by itself, its operands at hand, 620.)
// What did not help: two CTAs on one 256-row tile with the weights halved
// between them (their hand-over costs what the loads save), sixteen sum warps,
// 32 columns at a time (registers), longer scale runs in registers.  What did:
// the products' operands in uniform registers, shared memory addressed as
// such, no cluster-scope release on a barrier of every block, no exact
// division in the epilogue (its straight-line code cost more than a short k).
#include <cooperative_groups.h>

#include "bf16.cuh"
#include "check.h"
#include "coding.cuh"
#include "launch.h"
#include "plan.h"
#include "tc.cuh"
#include "thin.h"
#include "tilemap.h"
#include "trace.h"

namespace moe {

namespace cg = cooperative_groups;

constexpr int kBlk = 128;                    // k block, scale block, half of a tile's columns
constexpr int kBoxRows = 32;                 // rows of one TMA load of a: a group's last tile
                                             // loads no more than it has, rounded up to 32
constexpr int kStages = 4;
constexpr int kStageBytes = 3 * kTileRows * kBlk;  // a, first and second weight block
constexpr int kSumWarps = 8, kTmaWarp = 8, kMmaWarp = 9, kScaleWarp = 10, kScaleWarps = 2;
// Twelve warps are launched with 168 registers a thread; the sum warps, which
// hold 128 sums each thread, then take more and the others keep less, 384 * 168
// in all at most.  Which split compiles to the better loop was measured: without
// the activation 232 and 40 (dense 8191 x 7168 x 7168 308 us; 329 at 200 and 96,
// 336 at 192 and 112), with it 200 and 96 (prefill 777 us; 795 at 208 and 88, 914
// at 232 and 40, where the loops of the other warps spill).
__host__ __device__ constexpr int sum_regs(bool swiglu) { return swiglu ? 200 : 232; }
__host__ __device__ constexpr int other_regs(bool swiglu) { return swiglu ? 96 : 40; }
static_assert(256 * sum_regs(true) + 128 * other_regs(true) <= 384 * 168, "registers at launch");
static_assert(256 * sum_regs(false) + 128 * other_regs(false) <= 384 * 168, "registers at launch");
constexpr int kProductThreads = 32 * 12;
constexpr int kStageOut = 32 * 64;           // a sum warp's output staging: 32 rows of 64 bytes

// Two warps bring the scales of runs of four k blocks to shared memory, two runs
// ahead at most, by 4-byte asynchronous copies (a row's scales lie one after
// another, whatever their alignment).
constexpr int kScaleRun = 4;

struct Product {
    int N, E, cap, n, k;
    int wide;  // column blocks of a tile (1 or 2)
    const float *a_s;
    const int32_t *grp_off;
    const float *w_s;
    uint16_t *y;
    uint8_t *h_q;
    float *h_s;
    int32_t *status;
};

// First row and row count of expert e within its rank's rows, clipped.
__device__ __forceinline__ int2 group_rows(const Product &p, int e) {
    if (!p.grp_off) return make_int2(0, p.cap);
    const int Er = p.E / p.N, r = e / Er, j = e - r * Er;
    const int32_t *off = p.grp_off + (size_t)r * (Er + 1) + j;
    const int b = min(max(__ldg(off), 0), p.cap), t = min(max(__ldg(off + 1), b), p.cap);
    return make_int2(b, t - b);
}

struct Tile {
    int e, rows;      // expert; rows of the tile, 1 .. 128
    long long row0;   // first row, over all ranks
    int blk0, blk1;   // column blocks of 128; blk1 < 0: there is none
};

// Shared memory behind the stages and the output staging.
struct alignas(16) ProductShared {
    float rscale[2][kScaleRun][kTileRows], wscale[2][kScaleRun][2];
    uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], sfull[2], sempty[2], drain;
    uint32_t tmem;
    int stop, total;
    int wsum[32];
    uint32_t peak[2][kTileRows];
    int first[MOE_MAX_EXPERTS + 1];  // tiles of rows before each expert
};

constexpr size_t kProductSmem =
    1024 + (size_t)kStages * kStageBytes + (size_t)kSumWarps * kStageOut + sizeof(ProductShared);
static_assert(kProductSmem <= 232448, "a CTA's shared memory");

// Tiles run row tile first within runs of kRun row tiles, so that the CTAs at
// work at one time share weights and rows in L2.
constexpr int kRun = 16;

template <bool kSwiglu>
__device__ __forceinline__ Tile tile_at(const Product &p, const int *first, int ntn, int t) {
    int lo = 0, hi = p.E;  // first[lo] * ntn <= t < first[hi] * ntn
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] * ntn <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int mt = first[lo + 1] - first[lo], u = t - first[lo] * ntn;
    const int run = u / (kRun * ntn), width = min(kRun, mt - run * kRun);
    const int v = u - run * kRun * ntn, ni = v / width, mi = run * kRun + v - ni * width;
    const int2 g = group_rows(p, lo);
    Tile tile;
    tile.e = lo;
    tile.rows = min(kTileRows, g.y - mi * kTileRows);
    tile.row0 = (long long)(lo / (p.E / p.N)) * p.cap + g.x + mi * kTileRows;
    const int nb = p.n >> 7;
    if (kSwiglu) {
        tile.blk0 = ni;
        tile.blk1 = ni + (nb >> 1);
    } else {
        tile.blk0 = p.wide * ni;
        tile.blk1 = p.wide == 2 && 2 * ni + 1 < nb ? 2 * ni + 1 : -1;
    }
    return tile;
}

// Writes 64 bytes of each of the warp's 32 rows (v: a lane's own row) to
// dst + row * pitch, rows < rows only: through shared memory, so that four
// lanes write a row's 64 bytes together.
__device__ __forceinline__ void store_rows64(uint8_t *stage, const uint32_t (&v)[16], uint8_t *dst,
                                             size_t pitch, int rows) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j)  // 16-byte chunk j of row `lane`, swizzled by row
        *reinterpret_cast<uint4 *>(stage + lane * 64 + ((j ^ (lane >> 1)) & 3) * 16) =
            make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), j = lane & 3;
        if (r < rows)
            *reinterpret_cast<uint4 *>(dst + (size_t)r * pitch + j * 16) =
                *reinterpret_cast<const uint4 *>(stage + r * 64 + ((j ^ (r >> 1)) & 3) * 16);
    }
}

// kSplit, for few tiles: the two CTAs of a cluster share one tile, each with half
// of k; then each adds the other's sums for half of the rows and stores those (or
// none where either gave up).
template <bool kSwiglu, bool kSplit>
__global__ void __launch_bounds__(kProductThreads, 1)
    k_product(const Product p, const __grid_constant__ CUtensorMap map_a,
              const __grid_constant__ CUtensorMap map_w) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *stages = smem_raw + align1024(smem_raw);
    uint8_t *staging = stages + kStages * kStageBytes;
    ProductShared &s = *reinterpret_cast<ProductShared *>(staging + kSumWarps * kStageOut);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], kSumWarps);
            mbar_init(&s.sfull[i], kScaleWarps * 32);
            mbar_init(&s.sempty[i], kSumWarps);
        }
        mbar_init(&s.drain, 1);
        s.stop = 0;
        s.first[0] = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tc_alloc<512>(&s.tmem);
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_w);
    }
    // what is above runs while the kernel before this one ends
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    // row tiles before each expert
    int before = 0;
    for (int e0 = 0; e0 < p.E; e0 += kProductThreads) {
        const int e = e0 + tid;
        const int mt = e < p.E ? (group_rows(p, e).y + kTileRows - 1) / kTileRows : 0;
        const int upto = block_inclusive_scan(mt, s.wsum, &s.total);
        if (e < p.E) s.first[e + 1] = before + upto;
        before += s.total;
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile int *stop = &s.stop;
    const int nb = p.n >> 7, ntn = kSwiglu || p.wide == 2 ? (nb + 1) >> 1 : nb;
    // kSplit: a cluster has one tile at most (offsets that do not ascend may name
    // rows twice, and so more tiles than the grid was made for)
    const int Kb = p.k >> 7;
    const int tiles = kSplit ? min(before * ntn, (int)gridDim.x) : before * ntn;
    const int parts = kSplit ? gridDim.z : 1, part = kSplit ? blockIdx.z : 0;
    const int kb0 = kSplit ? Kb * part / parts : 0, kb1 = kSplit ? Kb * (part + 1) / parts : Kb;

    int issued = 0;  // k blocks whose loads are under way (TMA warp)
    if (warp >= kSumWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(other_regs(kSwiglu)));
        const uint32_t one = elect_one();  // the lane that loads, and that issues products
        if (warp == kTmaWarp) {
            bool ok = true;
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const Tile tile = tile_at<kSwiglu>(p, s.first, ntn, t);
                const int boxes = (tile.rows + kBoxRows - 1) / kBoxRows;
                const bool two = tile.blk1 >= 0;
                const uint32_t bytes = boxes * kBoxRows * kBlk + (two ? 2 : 1) * kBlk * kBlk;
                const int w0 = tile.e * p.n + tile.blk0 * kBlk, w1 = tile.e * p.n + tile.blk1 * kBlk;
#pragma unroll 1
                for (int b = kb0; b < kb1; ++b, ++issued) {
                    const int st = issued % kStages;
                    if (issued >= kStages &&
                        !(ok = wait_or_stop(&s.empty[st], (issued / kStages - 1) & 1, stop)))
                        break;
                    if (!one) continue;
                    uint8_t *a = stages + st * kStageBytes, *w = a + kTileRows * kBlk;
                    mbar_arrive_expect_tx(&s.full[st], bytes);
                    tma_tile(w, &map_w, b * kBlk, w0, &s.full[st]);
                    if (two) tma_tile(w + kBlk * kBlk, &map_w, b * kBlk, w1, &s.full[st]);
#pragma unroll 1
                    for (int i = 0; i < boxes; ++i)
                        tma_tile(a + i * kBoxRows * kBlk, &map_a, b * kBlk,
                                 (int)tile.row0 + i * kBoxRows, &s.full[st]);
                }
            }
        }
        if (warp == kMmaWarp) {
            bool ok = true;
            int it = 0;
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const Tile tile = tile_at<kSwiglu>(p, s.first, ntn, t);
                const uint32_t idesc =
                    tile.blk1 >= 0 ? tc_e4m3_f32(kTileRows, 256) : tc_e4m3_f32(kTileRows, 128);
#pragma unroll 1
                for (int b = kb0; b < kb1; ++b, ++it) {
                    const int st = it % kStages, ac = it & 1;
                    if (it >= 2 && !(ok = wait_or_stop(&s.tempty[ac], (it / 2 - 1) & 1, stop))) break;
                    if (!(ok = wait_or_stop(&s.full[st], (it / kStages) & 1, stop))) break;
                    tc_fence_after();
                    const uint64_t a = tc_operand(stages + st * kStageBytes);
                    const uint64_t w = tc_operand(stages + st * kStageBytes + kTileRows * kBlk);
#pragma unroll
                    for (int kk = 0; kk < kBlk / 32; ++kk)  // 32 bytes along k: 2 address units
                        tc_mma(tmem + ac * 256, a + kk * 2, w + kk * 2, idesc, kk > 0, one);
                    tc_commit(&s.empty[st], one);
                    tc_commit(&s.tfull[ac], one);
                }
            }
        }
        if (warp >= kScaleWarp) {
            bool ok = true;
            int run = 0;
            const int r = tid - kScaleWarp * 32;  // and r + 64; r < 8: a weight scale too
#pragma unroll 1
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const Tile tile = tile_at<kSwiglu>(p, s.first, ntn, t);
                // rows past the group's last take its scale; they are not stored
                const int r0 = min(r, tile.rows - 1), r1 = min(r + 64, tile.rows - 1);
                const float *as = p.a_s + (size_t)(tile.row0 + r0) * Kb;
                const int more = (r1 - r0) * Kb;
                const float *ws =
                    p.w_s + ((size_t)tile.e * nb + ((r & 1) && tile.blk1 >= 0 ? tile.blk1 : tile.blk0)) * Kb;
#pragma unroll 1
                for (int b = kb0; b < kb1; b += kScaleRun, ++run) {
                    const int buf = run & 1;
                    if (run >= 2)
                        ok = __all_sync(kFull, wait_or_stop(&s.sempty[buf], (run / 2 - 1) & 1, stop));
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < kScaleRun; ++i) {
                        const float *at = as + min(b + i, Kb - 1);
                        copy4_async(&s.rscale[buf][i][r], at);
                        copy4_async(&s.rscale[buf][i][r + 64], at + more);
                    }
                    if (r < 2 * kScaleRun)
                        copy4_async(&s.wscale[buf][r >> 1][r & 1], ws + min(b + (r >> 1), Kb - 1));
                    copies_arrive(&s.sfull[buf]);
                }
            }
            copies_wait();
        }
        if constexpr (kSplit) {
            __syncwarp();
            if ((int)blockIdx.x < tiles) {  // the sum warps' two
                cg::this_cluster().sync();
                // where the other CTA gave up its sums are not whole
                if (tid == kTmaWarp * 32 && *cg::this_cluster().map_shared_rank(&s.stop, 1 - part))
                    *stop = 1;
                __syncwarp();
                cg::this_cluster().sync();
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(sum_regs(kSwiglu)));
        const int quad = warp & 3, wg = warp >> 2;  // lanes 32 quad ..; columns 64 wg .. of each half
        const uint32_t mine = tmem + ((uint32_t)(quad * 32) << 16) + wg * 64;
        uint8_t *stage = staging + warp * kStageOut;
        bool ok = true;
        int it = 0, run = -1;
#pragma unroll 1
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const Tile tile = tile_at<kSwiglu>(p, s.first, ntn, t);
            const int r = quad * 32 + lane;
            const bool two = kSwiglu || tile.blk1 >= 0;
            uint64_t acc[2][32] = {};
#pragma unroll 1
            for (int b = kb0; b < kb1; ++b, ++it) {
                const int ac = it & 1, at = (b - kb0) % kScaleRun;
                if (at == 0) {
                    ++run;
                    ok = __all_sync(kFull, wait_or_stop(&s.sfull[run & 1], (run / 2) & 1, stop));
                    if (!ok) break;
                }
                const float sa = s.rscale[run & 1][at][r];
                const float2 sw = *reinterpret_cast<const float2 *>(s.wscale[run & 1][at]);
                const float f[2] = {sa * sw.x, sa * sw.y};
                ok = __all_sync(kFull, wait_or_stop(&s.tfull[ac], (it / 2) & 1, stop));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 8; ++c) {  // 16 columns
                    if (c == 4 && !two) break;
                    uint32_t v[16];
                    tc_ld16(v, mine + ac * 256 + c / 4 * 128 + c % 4 * 16);
                    tc_wait_ld();
                    if (c == 7 || (c == 3 && !two)) {  // all of it is in registers: the accumulator is free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&s.tempty[ac]);
                            if (at == kScaleRun - 1 || b == kb1 - 1) mbar_arrive(&s.sempty[run & 1]);
                        }
                    }
                    const uint64_t ff = pack2(__float_as_uint(f[c / 4]), __float_as_uint(f[c / 4]));
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        acc[c / 4][c % 4 * 8 + j] =
                            fma2(pack2(v[2 * j], v[2 * j + 1]), ff, acc[c / 4][c % 4 * 8 + j]);
                }
            }
            // either every sum warp has its sums or none goes on: the barriers
            // below are met by all
            ok = bar_named_all(1, kSumWarps * 32, ok);
            if constexpr (kSplit) {
                // the stages are free: [warp][column][lane]
                cg::cluster_group cluster = cg::this_cluster();
                float *left = reinterpret_cast<float *>(stages) + warp * 128 * 32 + lane;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const float2 f = unpack2(acc[i / 32][i % 32]);
                    left[2 * i * 32] = f.x;
                    left[(2 * i + 1) * 32] = f.y;
                }
                cluster.sync();
                // over `parts` though it is 2: without the loop it spills (22.2 us for 18.0,
                // 128 rows by 7168 x 7168)
                const bool mine = quad * parts / 4 == part;
                for (int q = 0; mine && q < parts; ++q) {
                    if (q == part) continue;
                    const float *o = cluster.map_shared_rank(left, q);
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        const float2 f = unpack2(acc[i / 32][i % 32]);
                        acc[i / 32][i % 32] = pack2(__float_as_uint(f.x + o[2 * i * 32]),
                                                    __float_as_uint(f.y + o[(2 * i + 1) * 32]));
                    }
                }
                cluster.sync();  // no CTA goes while it is read
                if (!mine || *stop) break;
            }
            if (!ok) break;
            const int rows = tile.rows - quad * 32;  // of this warp
            if constexpr (!kSwiglu) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1 && !two) break;
                    const int blk = h ? tile.blk1 : tile.blk0;
                    uint16_t *y = p.y + (size_t)(tile.row0 + quad * 32) * p.n + blk * 128 + wg * 64;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t o[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 f = unpack2(acc[h][q * 16 + i]);
                            o[i] = pack_bf16x2(f.x, f.y);
                        }
                        store_rows64(stage, o, reinterpret_cast<uint8_t *>(y + q * 32),
                                     (size_t)p.n * 2, rows);
                    }
                }
            } else {
                uint32_t am = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 g = unpack2(acc[0][i]), u = unpack2(acc[1][i]);
                    const float h0 = silu_mul(g.x, u.x), h1 = silu_mul(g.y, u.y);
                    am = max(am, max(abs_bits(h0), abs_bits(h1)));
                    acc[0][i] = pack2(__float_as_uint(h0), __float_as_uint(h1));
                }
                // the other 64 columns of the row's block are the other group's
                s.peak[wg][r] = am;
                bar_named(2 + quad, 64);  // the two warps of these rows
                const float scale = block_scale(max(s.peak[0][r], s.peak[1][r]));
                bar_named(2 + quad, 64);
                float inv = __frcp_rn(scale);
                if (scale < kTinyScale) {
                    // with scale 0 all to positive zeros, whose codes are zero bytes
                    const uint32_t by = __float_as_uint(scale == 0.0f ? 0.0f : kTinyUp);
                    const uint64_t up = pack2(by, by);
#pragma unroll
                    for (int i = 0; i < 32; ++i) acc[0][i] = fma2(acc[0][i], up, 0);
                    inv = scale == 0.0f ? 0.0f : __frcp_rn(scale * kTinyUp);
                }
                uint32_t o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 v0 = unpack2(acc[0][2 * i]), v1 = unpack2(acc[0][2 * i + 1]);
                    o[i] = code4_by(v0.x, v0.y, v1.x, v1.y, inv);
                }
                const int I = p.n >> 1;
                store_rows64(stage, o,
                             p.h_q + (size_t)(tile.row0 + quad * 32) * I + tile.blk0 * 128 + wg * 64,
                             (size_t)I, rows);
                if (wg == 0 && lane < rows)
                    p.h_s[(size_t)(tile.row0 + r) * (I >> 7) + tile.blk0] = scale;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (s.stop) {  // a kernel that gave up leaves no copy and no product in flight
        if (warp == kTmaWarp && lane == 0)
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait(&s.full[i % kStages], (i / kStages) & 1);
        if (warp == kMmaWarp) {
            tc_commit(&s.drain, elect_one());
            mbar_wait(&s.drain, 0);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kMmaWarp) tc_free<512>(tmem);
    if (tid == 0 && s.stop && p.status) flag(p.status, MOE_ST_TIMEOUT);
}

// ------------------------------------------------------------ host

static cudaError_t launch_product(Product p, const uint8_t *a_q, const uint8_t *w_q,
                                  cudaStream_t st) {
    const bool swiglu = p.h_q != nullptr;
    const ProductPlan plan = product_plan(p.N, p.cap, p.E, p.n, p.k, swiglu, sm_count());
    if (plan.few)
        return launch_thin_product(plan, p.N, p.E, p.cap, p.n, p.k, a_q, p.a_s, p.grp_off, w_q,
                                   p.w_s, p.y, p.h_q, p.h_s, p.status, st);
    CUtensorMap map_a, map_w;
    cudaError_t err = tile_map(&map_a, a_q, (int64_t)p.N * p.cap, p.k, kBoxRows);
    if (err == cudaSuccess) err = tile_map(&map_w, w_q, (int64_t)p.E * p.n, p.k, kBlk);
    if (err != cudaSuccess) return err;
    p.wide = plan.wide;
    const int parts = plan.parts;
    const auto kern = swiglu ? (parts > 1 ? k_product<true, true> : k_product<true, false>)
                             : (parts > 1 ? k_product<false, true> : k_product<false, false>);
    static LaunchMemo memo;
    int done = 0;
    err = memo.get(2 * swiglu + (parts > 1), &done, [&](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kProductSmem);
    });
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = (unsigned)parts;
    cfg.gridDim = dim3((unsigned)(plan.tiles < sm_count() ? plan.tiles : sm_count()), 1, (unsigned)parts);
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = kProductSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p, map_a, map_w);
}

// The checks that both products share; fills *p.
static int check_product(const moe_shape *sh, int64_t n, int k, const uint8_t *a_q,
                         const float *a_s, const int32_t *grp_off, const uint8_t *w_q,
                         const float *w_s, int32_t *status, Product *p) {
    moe_sizes z;
    int rc = moe_sizes_query(sh, &z);
    if (rc != MOE_OK) return rc;
    if ((rc = check_width(n)) != MOE_OK || (rc = check_width(k)) != MOE_OK) return rc;
    const int64_t rows = (int64_t)sh->N * z.cap;
    if (!ok_buffer(a_q, rows * k) || !ok_buffer(a_s, rows * (k / 128) * 4) ||
        !ok_buffer(w_q, sh->E * n * k) || !ok_buffer(w_s, 4) || !ok_optional(grp_off) ||
        !ok_optional(status))
        return MOE_EINVAL;
    if (!grp_off && sh->E != sh->N) return MOE_EINVAL;
    *p = Product{sh->N, sh->E, (int)z.cap, (int)n,  k,       2,     a_s,
                 grp_off, w_s, nullptr,    nullptr, nullptr, status};
    return MOE_OK;
}

}  // namespace moe

extern "C" int moe_expert_gemm(const moe_shape *sh, int n, int k, const uint8_t *a_q,
                               const float *a_s, const int32_t *grp_off, const uint8_t *w_q,
                               const float *w_s, uint16_t *y, int32_t *status, void *stream) {
    MOE_TRACE_CALL();
    moe::Product p;
    const int rc = moe::check_product(sh, n, k, a_q, a_s, grp_off, w_q, w_s, status, &p);
    if (rc != MOE_OK) return rc;
    if (!moe::ok_buffer(y, (int64_t)p.N * p.cap * n * 2)) return MOE_EINVAL;
    if (p.cap == 0) return MOE_OK;
    p.y = y;
    return moe::launch_product(p, a_q, w_q, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ECUDA;
}

extern "C" int moe_expert_gemm_swiglu(const moe_shape *sh, int inter, int k, const uint8_t *a_q,
                                      const float *a_s, const int32_t *grp_off,
                                      const uint8_t *w13_q, const float *w13_s, uint8_t *h_q,
                                      float *h_s, int32_t *status, void *stream) {
    MOE_TRACE_CALL();
    moe::Product p;
    int rc = moe::check_width(inter);
    if (rc != MOE_OK) return rc;
    rc = moe::check_product(sh, 2 * (int64_t)inter, k, a_q, a_s, grp_off, w13_q, w13_s, status, &p);
    if (rc != MOE_OK) return rc;
    const int64_t rows = (int64_t)p.N * p.cap;
    if (!moe::ok_buffer(h_q, rows * inter) || !moe::ok_buffer(h_s, rows * (inter / 128) * 4))
        return MOE_EINVAL;
    if (p.cap == 0) return MOE_OK;
    p.h_q = h_q;
    p.h_s = h_s;
    return moe::launch_product(p, a_q, w13_q, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ECUDA;
}
