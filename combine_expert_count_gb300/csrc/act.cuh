// act.cuh -- the activations of the 16-bit products (MOE_ACT_*), in fp32.
#pragma once

#include "common.cuh"

namespace moe {

// kExact: with the accurate exponential and division, for results that stay fp32;
// else the fast ones (about (|v| + 4) 2^-23 of the result off), for results that are
// rounded to bf16.  The error function is the complementary one and the tanh form a
// sigmoid, (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)), so that large negative v keep their
// digits.  Where exp(-v) overflows the quotient is 0.
template <bool kExact>
__device__ __forceinline__ float over_one_plus_exp(float v, float z) {  // v / (1 + exp(-z))
    if (kExact) return v / (1.0f + expf(-z));
    return __fdividef(v, 1.0f + __expf(-z));
}

template <bool kExact>
__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {
        case MOE_ACT_RELU: return v > 0.0f || v != v ? v : 0.0f;
        case MOE_ACT_SILU: return over_one_plus_exp<kExact>(v, v);
        case MOE_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678118654752f);
        case MOE_ACT_GELU_TANH:
            // 2 sqrt(2 / pi), and that times 0.044715
            return over_one_plus_exp<kExact>(
                v, v * __fmaf_rn(0.071354816272f, v * v, 1.5957691216057308f));
        case MOE_ACT_SIGMOID: return over_one_plus_exp<kExact>(1.0f, v);
        default: return v;
    }
}

}  // namespace moe
