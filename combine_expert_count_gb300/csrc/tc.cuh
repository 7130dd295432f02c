// tc.cuh -- inline-PTX wrappers for the tensor-core kernels (sm_103a): tiled
// TMA loads, tcgen05 products with their accumulators in tensor memory, packed
// fp32 arithmetic, and mbarrier waits that a stopped kernel leaves.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace moe {

// Bytes from p to the next multiple of 1024 in shared memory.  As an offset: a
// pointer rounded by itself would no longer be known to point there, and every
// access through it would be a generic one.
__device__ __forceinline__ uint32_t align1024(const void *p) { return -smem_addr(p) & 1023; }

// ------------------------------------------------------------ waits

// Where this holds for a thread, its waits below run out at once: a library that
// is compiled with it shows what a stopped kernel leaves.
#ifndef MOE_GIVE_UP
#define MOE_GIVE_UP false
#endif

// mbar_try_wait that may sleep up to 20 us before it answers: a waiting warp
// that asks again and again takes issue slots from those at work.
__device__ __forceinline__ bool mbar_try_wait_for(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}

// Waits for the phase with the given parity, at most about a second, and
// leaves at once when another role of the CTA has given up (*stop).  False:
// the phase did not complete; *stop is then set.
__device__ __forceinline__ bool wait_or_stop(uint64_t *bar, uint32_t parity, volatile int *stop) {
    if (MOE_GIVE_UP) {
        *stop = 1;
        return false;
    }
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (clock64() - t0 < kWaitCycles) {
        if (mbar_try_wait_for(bar, parity)) return true;
        if (*stop) return false;
    }
    *stop = 1;
    return false;
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// ------------------------------------------------------------ TMA

// Tile of a two-dimensional map at (x, y) -> shared memory; its bytes are
// counted on `bar`.  x is a multiple of 16 bytes.
__device__ __forceinline__ void tma_tile(void *dst, const CUtensorMap *map, int x, int y,
                                         uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ------------------------------------------------------------ small copies

// Four or sixteen bytes, global -> shared, asynchronously; `bar` gets this thread's arrival
// once its copies so far are there (an arrival that the barrier's count includes).
__device__ __forceinline__ void copy4_async(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copy16_async(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ------------------------------------------------------------ tcgen05

// Shared-memory operand: rows of 128 bytes along k, 128-byte swizzle, groups
// of eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t tc_operand(const void *p) {
    constexpr uint64_t kStride = (uint64_t)(1024 >> 4) << 32, kVersion = 1ull << 46,
                       kSwizzle128 = 2ull << 61;
    return (uint64_t)((smem_addr(p) & 0x3ffff) >> 4) | (1ull << 16) | kStride | kVersion |
           kSwizzle128;
}

// Instruction word of a k-major e4m3 x e4m3 -> fp32 product of M x N.
__host__ __device__ constexpr uint32_t tc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 1 in one lane of the (whole) warp, 0 in the others.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, e;\n\t}"
        : "=r"(one));
    return one;
}

// d (+)= a b^T over 32 elements of k, issued where `on`.  The whole warp comes
// here with `on` in one lane: a branch around the instruction would keep its
// operands out of the uniform registers, and four products with their waits and
// commits then take the warp 485 cycles to issue, not 239.
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate, uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(on)
        : "memory");
}

// `bar` gets one arrival once the thread's products so far are done (where `on`).
__device__ __forceinline__ void tc_commit(uint64_t *bar, uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_addr(bar)),
        "r"(on)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// kCols columns of the SM's tensor memory (a power of two from 32 to 512); one
// warp allocates and frees.
template <int kCols>
__device__ __forceinline__ void tc_alloc(uint32_t *where) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(where)),
                 "n"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int kCols>
__device__ __forceinline__ void tc_free(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(kCols));
}

// 16 columns of the warp's 32 lanes, one lane's row a thread.  The values are
// there after tc_wait_ld.
__device__ __forceinline__ void tc_ld16(uint32_t (&v)[16], uint32_t taddr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tc_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Makes this thread's shared-memory stores visible to the tensor cores and TMA.
__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ------------------------------------------------------------ packed fp32

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
// Two fused multiply-adds in one instruction.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Barrier `id` of `n` threads.
__device__ __forceinline__ void bar_named(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// The same; true where it is true for all of them.
__device__ __forceinline__ bool bar_named_all(int id, int n, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.and.aligned.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(id), "r"(n), "r"((uint32_t)ok)
        : "memory");
    return all != 0;
}

}  // namespace moe
