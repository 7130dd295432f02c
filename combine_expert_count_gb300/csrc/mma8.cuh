// mma8.cuh -- the warp-level e4m3 product and the activation of the experts'
// kernels.
#pragma once

#include "common.cuh"

namespace moe {

// c[16 x 8] += a[16 x 32] b[32 x 8], e4m3 operands, fp32 sums.  With lane =
// 4 g + t: a[i] holds four bytes of row g + 8 (i & 1) at 4 t + 16 (i >> 1), b0
// and b1 four bytes of column g at 4 t and 4 t + 16; c[i] is row
// g + 8 (i >> 1), column 2 t + (i & 1).
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// silu(g) * u with the fast exponential and division (about (|g| + 4) 2^-23 of
// the result off; the sums g and u come with more).  For g below -87 the
// quotient is 0 where the formula has a value of magnitude 2^-119 or less.
__device__ __forceinline__ float silu_mul(float g, float u) {
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

}  // namespace moe
