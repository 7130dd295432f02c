// thin.cu -- products of the experts' weights with few rows: the kernels of
// moe_layer_few, and moe_expert_gemm / moe_expert_gemm_swiglu for few rows
// (by plan.h).  They are bound by reading the weights once.
//
// The weights are the 128-row operand of the tensor cores and the rows of x (or
// h) the narrow one of 16 columns: a product costs what its real rows cost,
// and a lane of tensor memory is an output feature.  A CTA owns one block of
// 128 outputs of one expert (its gate and its up block; or one block over a run
// of experts) and streams the weights' 16 KB tiles by TMA through a ring of
// shared memory.  Two warps put the rows' 128-byte pieces beside them, a k block
// each in turn: by asynchronous copies as deep as the ring, or coded from x where
// the tokens are very few.  One warp issues the products of a k block; four add it,
// times its scales, to fp32 sums.  Two CTAs fit an SM, so one streams while the other
// starts or ends; together they keep about 200 KB of weights on the way.  Rows that
// come through registers, by four warps a block, are late where there are many: 64
// tokens on 64 experts (hidden 7168, experts of 2048) 521 us, now 415 to 420.
// Where there are fewer units than that, the CTAs of a cluster share each one's k
// blocks (thin_parts), and then its rows: each adds up and stores its own of them.
//
// Measured, hidden 7168, experts of 2048, top-8: four tokens of 256 experts 208 to
// 221 us (30 to 32 experts' weights, 6.1 to 6.8 TB/s), 32 tokens on 64 experts 401
// to 411 us (6.8 to 6.9 TB/s, a copy's rate).  One token, hidden 2048, experts of
// 768: 16.7 us (14.0 where L2 has the weights), of which they are 5.6 at a copy's
// rate; the rest is two launches, finding the rows (1 us each), the first blocks' way
// from HBM (1 us each) and the clusters' barriers.  The same layer on warp-level
// products (mma.sync, weights loaded straight to registers) took 311 and 1446 us
// for four tokens and 32: an e4m3 mma.sync is a score of instructions here, 340 a
// 2 KB tile in all, against 160 a 16 KB tile.
#include <cooperative_groups.h>

#include "bf16.cuh"
#include "check.h"
#include "coding.cuh"
#include "launch.h"
#include "tc.cuh"
#include "thin.h"
#include "tilemap.h"
#include "trace.h"

namespace moe {

namespace cg = cooperative_groups;

// What a kernel multiplies and what becomes of it:
//   kUp    rows coded from x, gate and up, activation coded to h     (few tokens)
//   kUpCoded  the same of rows that k_code_rows coded
//   kDown  rows of h, an output block of every token over all experts (few tokens)
//   kGemm, kSwiglu  grouped coded rows, as the entry points say
enum class Thin { kUp, kUpCoded, kDown, kGemm, kSwiglu };

// Warps 0-3 have the sums; the last two bring the rows, in turn: no more warps than
// stages, or one could miss two phases of a stage's barrier.  Eight warps leave two
// CTAs 128 registers a thread.
constexpr int kThinTma = 4, kThinMma = 5, kRowWarp = 6, kRowWarps = 2;
constexpr int kThinWarps = kRowWarp + kRowWarps, kThinThreads = 32 * kThinWarps;
constexpr int kTileBytes = 128 * 128;

struct ThinArgs {
    // few tokens
    int ntok, E, R, H, inter;
    bool by_expert;  // gate and up: units are experts, not assignments
    int passes;      // units of 16 rows that an expert may need
    const uint16_t *x;
    const int32_t *idx;
    const float *topk_w;
    uint8_t *h_q;
    float *h_s;
    uint16_t *out;
    // grouped rows
    int N, cap;
    const int32_t *grp_off;
    const uint8_t *a_q;
    const float *a_s;
    uint16_t *y;
    // both
    int n, k;  // outputs and inputs of the product
    const float *w_s;
    int32_t *status;
};

__host__ __device__ constexpr bool thin_up(Thin m) { return m == Thin::kUp || m == Thin::kUpCoded; }
__host__ __device__ constexpr bool thin_pair(Thin m) { return thin_up(m) || m == Thin::kSwiglu; }

// Up to so many tokens the gate and up kernel codes the rows of x that it multiplies,
// each of its CTAs again; beyond, a kernel before it codes them once.  us: four
// tokens 15.8 and 16.1 (8 experts of 768, hidden 2048, in L2), 98.9 and 100.6 (32 of 2048,
// 4096); with room for eight rows eight tokens 18.1 and 16.1, and fewer tokens 2% more.
constexpr int kOwnRows = 4;

// Accumulators in tensor memory: an item's way from its products to its sums
// takes several times as long as the products of a few rows.
constexpr int kAccs = 4;

// Ring stages for which two CTAs fit an SM; kDown's lists of many tokens take two
// stages' room (64 tokens on 64 experts, hidden 7168: one an SM, its 224 CTAs were
// two waves and the layer took 746 us; 522 with three stages).
__host__ __device__ constexpr int thin_stages(Thin m) { return thin_pair(m) ? 3 : 5; }
constexpr int kDownFewStages = 3;
__host__ __device__ constexpr int thin_stage_bytes(Thin m) {
    return (thin_pair(m) ? 2 : 1) * kTileBytes + kThinRowsAt * 128;
}

template <int kStages>
struct alignas(16) ThinShared {
    float scale[kStages][kThinRowsAt];  // of the rows' pieces in each stage
    uint64_t full[kStages], empty[kStages], tfull[kAccs], tempty[kAccs], drain;
    uint32_t tmem;
    int stop, total, unit[3];
    unsigned chosen[2];
    int wsum[32];
    int list[MOE_FEW_MAX_TOKENS];  // gate and up of few tokens: the expert's assignments,
    int token[MOE_FEW_MAX_TOKENS];  // one a token; and their tokens
};

template <Thin kMode, int kStages>
constexpr size_t thin_fixed_smem() {
    return 1024 + (size_t)kStages * thin_stage_bytes(kMode) + sizeof(ThinShared<kStages>);
}

// kDown's lists behind that: the sums [ntok][128]; ids; the lists' assignments
// and weights; for each expert its tokens as 64 bits and its first list place;
// the entries (an expert and up to 16 of its tokens): their experts and where
// their lists start.
__host__ __device__ constexpr int thin_entries(int A, int E) { return E + A / kThinRowsAt + 1; }
__host__ __device__ constexpr size_t thin_lists_smem(int ntok, int E, int R) {
    return (size_t)ntok * 512 + (size_t)ntok * R * 12 +
           ((size_t)3 * E + 2 * thin_entries(ntok * R, E)) * 4;
}

// Where byte 16 c of row r of a 128-byte-swizzled tile is.
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    return (uint32_t)r * 128 + (uint32_t)((c ^ (r & 7)) << 4);
}

// The maximum of a block of 128, four values a lane, as bits.
__device__ __forceinline__ uint32_t warp_amax(float a, float b, float c, float d) {
    return __reduce_max_sync(kFull,
                             max(max(abs_bits(a), abs_bits(b)), max(abs_bits(c), abs_bits(d))));
}

// One row's block of x: a lane's codes, and the scale.
__device__ __forceinline__ uint32_t code_row(float a, float b, float c, float d, float *scale) {
    *scale = block_scale(warp_amax(a, b, c, d));
    return *scale == 0.0f ? 0u : code4(a, b, c, d, *scale);
}

// Codes x's blocks of 128, a warp each, to where the layer's output will be: 128
// codes and the scale in the 256 bytes that the block's outputs take (so x and out
// may be the same).
constexpr int kCodedBlock = 256, kCodeWarps = 4;
__global__ void __launch_bounds__(32 * kCodeWarps)
    k_code_rows(int blocks, const uint16_t *x, uint8_t *out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int i = blockIdx.x * kCodeWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (i >= blocks) return;
    const uint2 w = *reinterpret_cast<const uint2 *>(x + (size_t)i * 128 + lane * 4);
    float scale;
    const uint32_t code =
        code_row(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y), &scale);
    uint8_t *to = out + (size_t)i * kCodedBlock;
    *reinterpret_cast<uint32_t *>(to + lane * 4) = code;
    if (lane == 0) *reinterpret_cast<float *>(to + 128) = scale;
}

template <Thin kMode, int kStages>
__global__ void __launch_bounds__(kThinThreads, 2)
    k_thin(const ThinArgs p, const __grid_constant__ CUtensorMap map_w) {
    constexpr bool kPair = thin_pair(kMode);
    constexpr int kHalves = kPair ? 2 : 1;
    constexpr int kBytes = thin_stage_bytes(kMode);
    constexpr int NMAX = kThinRowsAt;
    constexpr int kCols = kAccs * kHalves * NMAX;
    using Shared = ThinShared<kStages>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + align1024(smem_raw);
    Shared &s = *reinterpret_cast<Shared *>(ring + kStages * kBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blk = blockIdx.x, Kb = p.k >> 7, nb = p.n >> 7;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();

    // ---------------------------------------------------------------- set-up
    // while the kernel before this one ends
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], kMode == Thin::kUp ? 2 : 1 + 32);  // TMA's, and a row warp's
            mbar_init(&s.empty[i], 1 + 4);
        }
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 4);
        }
        mbar_init(&s.drain, 1);
        s.stop = 0;
        fence_mbar_init();
        tma_prefetch_map(&map_w);
    }
    if (warp == kThinMma) tc_alloc<kCols>(&s.tmem);
    // the kernel before kUpCoded and kDown is this call's, which has waited: only
    // what it made is waited for, where it is read
    constexpr bool kLate = kMode == Thin::kDown || kMode == Thin::kUpCoded;
    if constexpr (!kLate) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const auto leave = [&]() {  // nothing to do: all threads
        __syncthreads();
        if (warp == kThinMma) tc_free<kCols>(s.tmem);
        // not done before the kernel that it follows is
        if constexpr (kLate) asm volatile("griddepcontrol.wait;" ::: "memory");
    };

    // ---------------------------------------------------------------- the unit
    // kDown: the whole list of experts; else one expert and its m rows
    int e = 0, m = 0;
    long long row0 = 0;
    float *sums = reinterpret_cast<float *>(&s + 1);  // kDown, [ntok][128]
    int *ids = reinterpret_cast<int *>(sums + (kMode == Thin::kDown ? p.ntok * 128 : 0));
    const int A = p.ntok * p.R;
    int *slot = ids + A;  // lists of assignments
    float *weight = reinterpret_cast<float *>(slot + A);
    unsigned *who = reinterpret_cast<unsigned *>(weight + A);  // [E][2]
    int *place = reinterpret_cast<int *>(who + 2 * p.E), *start = place + p.E;
    int *experts = start + thin_entries(A, p.E);
    int r0 = 0;  // the unit's first row of its expert's
    int U = 0;  // kDown: entries
    if constexpr (thin_up(kMode)) {
        // CTAs with the same weights and other rows are neighbours: one reads HBM, the
        // others L2 (16 experts, 64 tokens, 16 rows an expert on average, hidden 7168: 146
        // us; 158 with all experts' first 16 rows first; 8 experts with 8 rows at most 17.6
        // and 17.0)
        const int unit = blockIdx.y / p.passes;
        r0 = blockIdx.y % p.passes * NMAX;
        ids = reinterpret_cast<int *>(ring);  // the ring is not in use yet
        int bad = 0;
        for (int i = tid; i < A; i += kThinThreads) {
            ids[i] = p.idx[i];
            bad |= (unsigned)ids[i] >= (unsigned)p.E;
        }
        if (blockIdx.x == 0 && blockIdx.y == 0 && part == 0) {
            bad = __syncthreads_or(bad);
            if (tid == 0) *p.status = bad ? MOE_ST_BAD_EXPERT : 0;
        }
        __syncthreads();
        e = p.by_expert ? unit : ids[unit];
        if ((unsigned)e >= (unsigned)p.E) return leave();
        // thread t < 64: token t's first assignment to the expert
        int k = -1;
        if (tid < MOE_FEW_MAX_TOKENS) {
            if (tid < p.ntok)
                for (int i = p.R - 1; i >= 0; --i)
                    if (ids[tid * p.R + i] == e) k = i;
            const unsigned got = __ballot_sync(kFull, k >= 0);
            if (lane == 0) s.chosen[warp] = got;
        }
        __syncthreads();
        const unsigned lo = s.chosen[0], hi = s.chosen[1];
        m = __popc(lo) + __popc(hi);
        if (k >= 0) {
            const unsigned below = (1u << lane) - 1u;
            const int at = warp == 0 ? __popc(lo & below) : __popc(lo) + __popc(hi & below);
            s.list[at] = tid * p.R + k;
            s.token[at] = tid;
        }
        __syncthreads();
        if (m <= r0 || (!p.by_expert && s.list[0] != unit)) return leave();
        m = min(m - r0, NMAX);
    } else if constexpr (kMode == Thin::kDown) {
        for (int i = tid; i < 2 * p.E; i += kThinThreads) who[i] = 0;
        for (int i = tid; i < p.ntok * 128; i += kThinThreads) sums[i] = 0.0f;
        for (int i = tid; i < A; i += kThinThreads) ids[i] = p.idx[i];
        __syncthreads();
        for (int i = tid; i < A; i += kThinThreads) {
            const int t = i / p.R;
            if ((unsigned)ids[i] < (unsigned)p.E)
                atomicOr(who + 2 * ids[i] + (t >> 5), 1u << (t & 31));
        }
        __syncthreads();
        int L = 0;
        for (int e0 = 0; e0 < p.E; e0 += kThinThreads) {
            // entries and list places before each expert's, in one scan
            const int x = e0 + tid;
            const int c = x < p.E ? __popc(who[2 * x]) + __popc(who[2 * x + 1]) : 0;
            const int both = ((c + NMAX - 1) / NMAX << 16) + c;
            const int upto = block_inclusive_scan(both, s.wsum, &s.total) - both;
            const int u = U + (upto >> 16), l = L + (upto & 0xffff);
            for (int i = 0; i * NMAX < c; ++i) {
                experts[u + i] = x;
                start[u + i] = l + i * NMAX;
            }
            if (c > 0) place[x] = l;
            U += s.total >> 16;
            L += s.total & 0xffff;
            __syncthreads();
        }
        if (tid == 0) start[U] = L;
        // an expert's tokens in their order: the parts of a cluster make the same lists
        for (int i = tid; i < A; i += kThinThreads) {
            const int x = ids[i], t = i / p.R;
            if ((unsigned)x >= (unsigned)p.E) continue;
            bool again = false;  // an earlier slot of the token has this expert
            for (int q = t * p.R; q < i; ++q) again |= ids[q] == x;
            if (again) continue;
            float w = 0.0f;
            for (int q = i; q < t * p.R + p.R; ++q)
                if (ids[q] == x) w += p.topk_w[q];
            const unsigned below = (1u << (t & 31)) - 1u;
            const int at = place[x] + (t < 32 ? __popc(who[2 * x] & below)
                                              : __popc(who[2 * x]) + __popc(who[2 * x + 1] & below));
            slot[at] = i;
            weight[at] = w;
        }
    } else {
        // the unit-th 16 rows of one expert
        if (tid == 0) s.unit[0] = -1;
        __syncthreads();
        int seen = 0;
        const int Er = p.E / p.N, unit = blockIdx.y;
        for (int e0 = 0; e0 < p.E; e0 += kThinThreads) {
            const int x = e0 + tid;
            int b = 0, c = 0;
            if (x < p.E && p.grp_off) {
                const int32_t *off = p.grp_off + (size_t)(x / Er) * (Er + 1) + x % Er;
                b = min(max(off[0], 0), p.cap);
                c = min(max(off[1], b), p.cap) - b;
            } else if (x < p.E) {
                c = p.cap;
            }
            const int mine = (c + NMAX - 1) / NMAX;
            const int before = seen + block_inclusive_scan(mine, s.wsum, &s.total) - mine;
            if (before <= unit && unit < before + mine) {
                s.unit[0] = x;
                s.unit[1] = b + (unit - before) * NMAX;
                s.unit[2] = c - (unit - before) * NMAX;
            }
            seen += s.total;
            __syncthreads();
        }
        e = s.unit[0];
        if (e < 0) return leave();
        m = min(s.unit[2], NMAX);
        row0 = (long long)(e / Er) * p.cap + s.unit[1];
    }

    fence_async_smem();  // gate and up: the ids lay where the ring is
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile int *stop = &s.stop;

    // The CTA's items, in order: k blocks b of (expert, rows).  kDown: a run of
    // all experts' blocks; else a run of the one expert's.
    const int all = kMode == Thin::kDown ? U * Kb : Kb;
    const int i0 = (int)((long long)all * part / parts);
    const int i1 = (int)((long long)all * (part + 1) / parts);
    int issued = 0;  // items whose loads are under way (TMA warp)

    float acc[kHalves][NMAX];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int j = 0; j < NMAX; ++j) acc[h][j] = 0.0f;

    if (warp == kThinTma) {
        const uint32_t one = elect_one();
        for (int item = i0; item < i1; ++item, ++issued) {
            const int u = kMode == Thin::kDown ? item / Kb : 0, b = item - u * Kb;
            const int ex = kMode == Thin::kDown ? experts[u] : e, st = issued % kStages;
            if (issued >= kStages && !wait_or_stop(&s.empty[st], (issued / kStages - 1) & 1, stop))
                break;
            if (!one) continue;
            uint8_t *w = ring + st * kBytes;
            mbar_arrive_expect_tx(&s.full[st], kHalves * kTileBytes);
            tma_tile(w, &map_w, b * 128, ex * p.n + blk * 128, &s.full[st]);
            if (kPair)
                tma_tile(w + kTileBytes, &map_w, b * 128, ex * p.n + (p.n >> 1) + blk * 128,
                         &s.full[st]);
        }
    } else if (warp == kThinMma) {
        const uint32_t one = elect_one(), idesc = tc_e4m3_f32(128, NMAX);
        int it = 0;
        for (int item = i0; item < i1; ++item, ++it) {
            const int st = it % kStages, ac = it % kAccs;
            if (it >= kAccs && !wait_or_stop(&s.tempty[ac], (it / kAccs - 1) & 1, stop)) break;
            if (!wait_or_stop(&s.full[st], (it / kStages) & 1, stop)) break;
            fence_async_smem();  // the rows, for the tensor cores
            tc_fence_after();
            const uint64_t w = tc_operand(ring + st * kBytes);
            const uint64_t rows = tc_operand(ring + st * kBytes + kHalves * kTileBytes);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 bytes along k: 2 address units
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    tc_mma(tmem + (ac * kHalves + h) * NMAX, w + h * (kTileBytes >> 4) + kk * 2,
                           rows + kk * 2, idesc, kk > 0, one);
            tc_commit(&s.empty[st], one);
            tc_commit(&s.tfull[ac], one);
        }
    } else if (warp >= kRowWarp) {
        const int rw = warp - kRowWarp;
        if constexpr (kMode == Thin::kUp) {
            // A warp codes its next item's rows before it waits for their stage, and loads
            // the ones after meanwhile.  A row is all lanes', four values each.
            const uint16_t *x[kOwnRows];
            uint2 v[kOwnRows];
            uint32_t code[kOwnRows];
            float scale[kOwnRows];
#pragma unroll
            for (int q = 0; q < kOwnRows; ++q) {
                if (q >= m || i0 + rw >= i1) break;
                x[q] = p.x + (size_t)s.token[q] * p.H + lane * 4;
                v[q] = *reinterpret_cast<const uint2 *>(x[q] + (i0 + rw) * 128);
            }
            for (int it = rw; i0 + it < i1; it += kRowWarps) {
                const int st = it % kStages, next = i0 + it + kRowWarps;
#pragma unroll
                for (int q = 0; q < kOwnRows; ++q) {
                    if (q >= m) break;
                    const float f0 = bf16_lo(v[q].x), f1 = bf16_hi(v[q].x), f2 = bf16_lo(v[q].y),
                                f3 = bf16_hi(v[q].y);
                    if (next < i1) v[q] = *reinterpret_cast<const uint2 *>(x[q] + next * 128);
                    code[q] = code_row(f0, f1, f2, f3, &scale[q]);
                }
                if (it >= kStages &&
                    !__all_sync(kFull, wait_or_stop(&s.empty[st], (it / kStages - 1) & 1, stop)))
                    break;
                uint8_t *rows = ring + st * kBytes + kHalves * kTileBytes;
#pragma unroll
                for (int q = 0; q < kOwnRows; ++q) {
                    if (q >= m) break;
                    *reinterpret_cast<uint32_t *>(rows + swizzled(q, lane >> 2) + (lane & 3) * 4) =
                        code[q];
                    if (lane == 0) s.scale[st][q] = scale[q];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.full[st]);
            }
        } else {
            // eight lanes a row, by asynchronous copies
            if constexpr (kLate) asm volatile("griddepcontrol.wait;" ::: "memory");
            // where the kernel that makes h gave up, this one does too
            const int before = kMode == Thin::kDown
                                   ? *reinterpret_cast<volatile const int32_t *>(p.status) : 0;
            const int c = lane & 7;
            for (int it = rw; i0 + it < i1; it += kRowWarps) {
                const int item = i0 + it, st = it % kStages;
                const int u = kMode == Thin::kDown ? item / Kb : 0, b = item - u * Kb;
                const int l = kMode == Thin::kDown ? start[u] : 0;
                const int mm = kMode == Thin::kDown ? start[u + 1] - l : m;
                if (it >= kStages &&
                    !__all_sync(kFull, wait_or_stop(&s.empty[st], (it / kStages - 1) & 1, stop)))
                    break;
                uint8_t *rows = ring + st * kBytes + kHalves * kTileBytes;
                for (int r = lane >> 3; r < mm; r += 4) {
                    const uint8_t *q;
                    const float *sc;
                    if constexpr (kMode == Thin::kUpCoded) {
                        q = p.a_q + ((size_t)s.token[r0 + r] * Kb + b) * kCodedBlock;
                        sc = reinterpret_cast<const float *>(q + 128);
                    } else {
                        const size_t row = kMode == Thin::kDown ? (size_t)slot[l + r] : row0 + r;
                        q = (kMode == Thin::kDown ? p.h_q : p.a_q) + row * p.k + b * 128;
                        sc = (kMode == Thin::kDown ? p.h_s : p.a_s) + row * Kb + b;
                    }
                    copy16_async(rows + swizzled(r, c), q + c * 16);
                    if (c == 0) copy4_async(&s.scale[st][r], sc);
                }
                copies_arrive(&s.full[st]);
            }
            copies_wait();
            if (before & MOE_ST_TIMEOUT) *stop = 1;
        }
    } else {
        // sums: lane = output 32 warp + lane of the block, column = row of x or h
        const uint32_t mine = tmem + ((uint32_t)(warp * 32) << 16);
        int it = 0;
        for (int item = i0; item < i1;) {
            const int u = kMode == Thin::kDown ? item / Kb : 0, b0 = item - u * Kb;
            const int end = min(i1, (u + 1) * Kb), ex = kMode == Thin::kDown ? experts[u] : e;
            if (kMode == Thin::kDown) m = start[u + 1] - start[u];
            const float *ws = p.w_s + ((size_t)ex * nb + blk) * Kb + b0;
            const float *wu = ws + (size_t)(kPair ? nb >> 1 : 0) * Kb;
            const int nblk = end - item;
            // weight scales two blocks ahead
            float g0 = __ldg(ws), g1 = __ldg(ws + min(1, nblk - 1));
            float u0 = __ldg(wu), u1 = __ldg(wu + min(1, nblk - 1));
            bool ok = true;
            for (int b = 0; b < nblk; ++b, ++it) {
                const int st = it % kStages, ac = it % kAccs;
                const float g2 = __ldg(ws + min(b + 2, nblk - 1));
                const float u2 = kPair ? __ldg(wu + min(b + 2, nblk - 1)) : 0.0f;
                // the rows' scales were stored before their arrivals on full
                ok = wait_or_stop(&s.tfull[ac], (it / kAccs) & 1, stop) &&
                     wait_or_stop(&s.full[st], (it / kStages) & 1, stop);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                tc_fence_after();
                uint32_t d[kHalves][NMAX];
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    tc_ld16(d[h], mine + (ac * kHalves + h) * NMAX);
                float sc[NMAX];
#pragma unroll
                for (int j = 0; j < NMAX / 4; ++j) {
                    const float4 f = *reinterpret_cast<const float4 *>(&s.scale[st][j * 4]);
                    sc[4 * j] = f.x;
                    sc[4 * j + 1] = f.y;
                    sc[4 * j + 2] = f.z;
                    sc[4 * j + 3] = f.w;
                }
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < NMAX; ++j) {
                    acc[0][j] = __fmaf_rn(sc[j] * g0, __uint_as_float(d[0][j]), acc[0][j]);
                    if (kPair)
                        acc[kHalves - 1][j] =
                            __fmaf_rn(sc[j] * u0, __uint_as_float(d[kHalves - 1][j]),
                                      acc[kHalves - 1][j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s.tempty[ac]);
                    mbar_arrive(&s.empty[st]);
                }
                g0 = g1;
                g1 = g2;
                u0 = u1;
                u1 = u2;
            }
            if (!ok) break;
            item = end;
            if constexpr (kMode == Thin::kDown) {
                // a thread owns its output of every token
#pragma unroll
                for (int j = 0; j < NMAX; ++j) {
                    if (j < m) {
                        const int at = start[u] + j;
                        float *t = sums + (slot[at] / p.R) * 128 + tid;
                        *t = __fmaf_rn(weight[at], acc[0][j], *t);
                    }
                    acc[0][j] = 0.0f;
                }
            }
        }
    }

    // ---------------------------------------------------------------- the end
    tc_fence_before();
    __syncthreads();
    if (s.stop) {  // a kernel that gave up leaves no copy and no product in flight
        if (warp == kThinTma && lane == 0)
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait(&s.full[i % kStages], (i / kStages) & 1);
        if (warp == kThinMma) {
            tc_commit(&s.drain, elect_one());
            mbar_wait(&s.drain, 0);
        }
        if (tid == 0 && p.status) flag(p.status, MOE_ST_TIMEOUT);
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kThinMma) tc_free<kCols>(tmem);

    // Where a part gave up, the sums are not whole and no part stores any.  Each
    // lane reads one part's flag; the answer is waited for where a warp has its sums
    // (0.1 us of one row's product by 7168 x 2048, 5.3 and 5.4; asked only where the
    // sums are the NaN that such a part would leave: gate/up over 128 experts 64.1, 61.9).
    const auto gave_up = [&]() { return ld_dsmem(dsmem_addr(&s.stop, min(lane, parts - 1))); };
    if constexpr (kMode == Thin::kDown) {
        // the parts of the experts' run, added in the cluster's order
        if (parts > 1) cluster.sync();
        const int any = gave_up();
        for (int i = part * kThinThreads + tid; i < p.ntok * 64; i += parts * kThinThreads) {
            float2 v = make_float2(0.0f, 0.0f);
            for (int q = 0; q < parts; ++q) {
                const float2 o =
                    *reinterpret_cast<const float2 *>(cluster.map_shared_rank(sums + i * 2, q));
                v.x += o.x;
                v.y += o.y;
            }
            if (__any_sync(kFull, any)) break;  // whole warps come here: 64 outputs a token
            uint16_t *to = p.out + (size_t)(i >> 6) * p.H + blk * 128 + (i & 63) * 2;
            *reinterpret_cast<uint32_t *>(to) = pack_bf16x2(v.x, v.y);
        }
        if (parts > 1) cluster.sync();  // no part goes while it is read
        return;
    }
    // The sums go through the ring, [half][row][128], so that a warp can take a row:
    // the row's block maximum is then its own, and the rows are shared by all warps of
    // all parts (which fetch what the others have of theirs).  A row after another
    // by the four warps with the sums was 0.2 us a row.
    float *left = reinterpret_cast<float *>(ring);
    if (warp < 4)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int j = 0; j < NMAX; ++j)
                if (j < m) left[(h * NMAX + j) * 128 + tid] = acc[h][j];
    if (parts > 1)
        cluster.sync();
    else
        __syncthreads();
    const int any = gave_up();
    for (int j = part + warp * parts; j < m; j += parts * kThinWarps) {
        float4 v[kHalves];
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const float *at = left + (h * NMAX + j) * 128 + lane * 4;
            v[h] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int q = 0; q < parts; ++q) {
                const float4 o = *reinterpret_cast<const float4 *>(
                    parts > 1 ? cluster.map_shared_rank(at, q) : at);
                v[h].x += o.x;
                v[h].y += o.y;
                v[h].z += o.z;
                v[h].w += o.w;
            }
        }
        if (__any_sync(kFull, any)) break;
        const size_t row = thin_up(kMode) ? (size_t)s.list[r0 + j] : (size_t)(row0 + j);
        if constexpr (!kPair) {
            *reinterpret_cast<uint2 *>(p.y + row * p.n + blk * 128 + lane * 4) =
                make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[0].z, v[0].w));
        } else {
            const float4 g = v[0], u = v[kHalves - 1];
            const float a = silu_mul(g.x, u.x), b = silu_mul(g.y, u.y), c = silu_mul(g.z, u.z),
                        d = silu_mul(g.w, u.w);
            const float scale = block_scale(warp_amax(a, b, c, d));
            float first;
            const float inv = code_factor(scale, &first);  // as the 128-row tiles code it
            const int I = p.n >> 1;
            *reinterpret_cast<uint32_t *>(p.h_q + row * I + blk * 128 + lane * 4) =
                scale == 0.0f ? 0u : code4_by(a * first, b * first, c * first, d * first, inv);
            if (lane == 0) p.h_s[row * (I >> 7) + blk] = scale;
        }
    }
    if (parts > 1) cluster.sync();  // no part goes while it is read
}

// ------------------------------------------------------------ host

constexpr int kMostSmem = 232448, kTwoSmem = 113 * 1024;  // a CTA's; of two an SM

template <Thin kMode, int kStages = thin_stages(kMode)>
static cudaError_t launch_thin(ThinArgs p, const CUtensorMap &map, dim3 grid, int parts,
                               size_t more_smem, cudaStream_t st) {
    constexpr size_t kFixed = thin_fixed_smem<kMode, kStages>();
    const auto kern = k_thin<kMode, kStages>;
    static_assert(kFixed <= kTwoSmem, "two CTAs an SM");
    static_assert(thin_fixed_smem<Thin::kDown, thin_stages(Thin::kDown)>() +
                          thin_lists_smem(MOE_FEW_MAX_TOKENS, MOE_MAX_EXPERTS, MOE_MAX_TOPK) <=
                      kMostSmem,
                  "a CTA's shared memory");
    static LaunchMemo memo;
    int done = 0;
    cudaError_t err = memo.get(0, &done, [&](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kMostSmem);
    });
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = (unsigned)parts;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    grid.z = (unsigned)parts;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThinThreads);
    cfg.dynamicSmemBytes = kFixed + more_smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p, map);
}

cudaError_t launch_thin_product(const ProductPlan &plan, int N, int E, int cap, int n, int k,
                                const uint8_t *a_q, const float *a_s, const int32_t *grp_off,
                                const uint8_t *w_q, const float *w_s, uint16_t *y, uint8_t *h_q,
                                float *h_s, int32_t *status, cudaStream_t st) {
    CUtensorMap map;
    cudaError_t err = tile_map(&map, w_q, (int64_t)E * n, k, 128);
    if (err != cudaSuccess) return err;
    ThinArgs p = {};
    p.E = E;
    p.N = N;
    p.cap = cap;
    p.grp_off = grp_off;
    p.a_q = a_q;
    p.a_s = a_s;
    p.w_s = w_s;
    p.y = y;
    p.h_q = h_q;
    p.h_s = h_s;
    p.n = n;
    p.k = k;
    p.status = status;
    const dim3 grid((unsigned)(h_q ? n >> 8 : n >> 7), (unsigned)plan.units);
    if (h_q) return launch_thin<Thin::kSwiglu>(p, map, grid, plan.parts, 0, st);
    return launch_thin<Thin::kGemm>(p, map, grid, plan.parts, 0, st);
}

static cudaError_t launch_code_rows(int blocks, const uint16_t *x, uint8_t *out, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((blocks + kCodeWarps - 1) / kCodeWarps));
    cfg.blockDim = dim3(32 * kCodeWarps);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_code_rows, blocks, x, out);
}

static cudaError_t launch_few(ThinArgs p, const uint8_t *w13_q, const float *w13_s,
                              const uint8_t *w2_q, const float *w2_s, cudaStream_t st) {
    if (p.ntok == 0) return cudaMemsetAsync(p.status, 0, 4, st);
    CUtensorMap up, down;
    cudaError_t err = tile_map(&up, w13_q, (int64_t)p.E * 2 * p.inter, p.H, 128);
    if (err == cudaSuccess) err = tile_map(&down, w2_q, (int64_t)p.E * p.H, p.inter, 128);
    if (err != cudaSuccess) return err;
    const int A = p.ntok * p.R;
    p.by_expert = A > p.E;
    p.passes = (p.ntok + kThinRowsAt - 1) / kThinRowsAt;
    const int units = p.by_expert ? p.E : A;
    const dim3 gup((unsigned)(p.inter >> 7), (unsigned)(units * p.passes));
    p.n = 2 * p.inter;
    p.k = p.H;
    p.w_s = w13_s;
    // an expert's second and further 16 rows are A / 16 units more at most
    const int64_t real = p.passes > 1 ? units + A / kThinRowsAt : units;
    const int up_parts = thin_parts((real < gup.y ? real : gup.y) * gup.x, p.H >> 7, sm_count());
    if (p.ntok <= kOwnRows) {
        err = launch_thin<Thin::kUp>(p, up, gup, up_parts, 0, st);
    } else {
        uint8_t *coded = reinterpret_cast<uint8_t *>(p.out);
        err = launch_code_rows(p.ntok * (p.H >> 7), p.x, coded, st);
        p.a_q = coded;
        if (err == cudaSuccess) err = launch_thin<Thin::kUpCoded>(p, up, gup, up_parts, 0, st);
    }
    if (err != cudaSuccess) return err;
    p.n = p.H;
    p.k = p.inter;
    p.w_s = w2_s;
    const dim3 gdown((unsigned)(p.H >> 7));
    const int parts = thin_parts(gdown.x, (int64_t)units * (p.inter >> 7), sm_count());
    const size_t lists = thin_lists_smem(p.ntok, p.E, p.R);
    constexpr size_t kFixed = thin_fixed_smem<Thin::kDown, thin_stages(Thin::kDown)>();
    if (kFixed + lists <= kTwoSmem) return launch_thin<Thin::kDown>(p, down, gdown, parts, lists, st);
    return launch_thin<Thin::kDown, kDownFewStages>(p, down, gdown, parts, lists, st);
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
    moe::ThinArgs p = {};
    p.ntok = (int)ntok;
    p.E = sh->E;
    p.R = sh->R;
    p.H = sh->H;
    p.inter = inter;
    p.x = x;
    p.idx = topk_idx;
    p.topk_w = topk_w;
    p.h_q = h_q;
    p.h_s = h_s;
    p.out = out;
    p.status = status;
    return moe::launch_few(p, w13_q, w13_s, w2_q, w2_s, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ECUDA;
}
