// act.cuh -- the activations of the 16-bit products (MOE_ACT_*), in fp32.
#pragma once

#include "common.cuh"

namespace moe {

// kExact: with the accurate exponential and division, for results that stay fp32;
// else the fast ones, for results that are rounded to bf16.  Those are about (1.2 |z| + 4)
// 2^-23 of the result off by the exponential of z and the division, and by z's own
// roundings: silu and sigmoid, z = v, no more; the tanh form, z = 1.6 v + 0.071 v^3, another
// 1.5 |z| 2^-23; the gelu, z = v^2 / 2, another 0.5 |z| 2^-23, its polynomial's roundings,
// 6 2^-23, and its fit, 2^-19 (for v > 0 less).  Where a bf16 result is not next to 0 these
// are 3e-5 or less, a hundredth of its half step.  The error function is the complementary one and the tanh form a
// sigmoid, (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)), so that large negative v keep their
// digits.  Where exp(-v) overflows the quotient is 0.
template <bool kExact>
__device__ __forceinline__ float over_one_plus_exp(float v, float z) {  // v / (1 + exp(-z))
    if (kExact) return v / (1.0f + expf(-z));
    return __fdividef(v, 1.0f + __expf(-z));
}

// The probability below v of a standard normal, whose product with v is the gelu:
// for v < 0 exp(-v^2 / 2) t P(t) with t = 1 / (1 + |v| / 5), else 1 minus that of -v.
// P is a polynomial of degree six fitted to exp(v^2 / 2) erfc(|v| / sqrt(2)) / (2 t)
// by least squares with weights that even out its relative error, over |v| from 0 to
// 14: at most 1.7e-6, 2^-19, in fp32.  The complementary error function itself takes
// twice the instructions, which a tile with a short k then waits for (512 x 9728 x 64:
// 15.9 us, 7.4 without an activation).
__device__ __forceinline__ float normal_below(float v) {
    const float a = fabsf(v), t = __fdividef(1.0f, __fmaf_rn(0.2f, a, 1.0f));
    float s = 0.27909577f;
    s = __fmaf_rn(s, t, -0.38683176f);
    s = __fmaf_rn(s, t, 0.44694775f);
    s = __fmaf_rn(s, t, -0.12319261f);
    s = __fmaf_rn(s, t, 0.13253959f);
    s = __fmaf_rn(s, t, 0.07109163f);
    s = __fmaf_rn(s, t, 0.08035023f);
    s *= t * __expf(-0.5f * a * a);
    return v > 0.0f ? 1.0f - s : s;
}

// One activation of all of v: its kind is asked once, so that only its code is fetched.
template <bool kExact, int n>
__device__ __forceinline__ void activate(int act, float (&v)[n]) {
    const auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = f(v[i]);
    };
    switch (act) {
        case MOE_ACT_RELU:
            return each([](float a) { return a > 0.0f || a != a ? a : 0.0f; });
        case MOE_ACT_SILU:
            return each([](float a) { return over_one_plus_exp<kExact>(a, a); });
        case MOE_ACT_GELU:
            return each([](float a) {
                return kExact ? 0.5f * a * erfcf(a * -0.70710678118654752f) : a * normal_below(a);
            });
        case MOE_ACT_GELU_TANH:  // 2 sqrt(2 / pi), and that times 0.044715
            return each([](float a) {
                return over_one_plus_exp<kExact>(
                    a, a * __fmaf_rn(0.071354816272f, a * a, 1.5957691216057308f));
            });
        case MOE_ACT_SIGMOID:
            return each([](float a) { return over_one_plus_exp<kExact>(1.0f, a); });
        default: return;
    }
}

}  // namespace moe
