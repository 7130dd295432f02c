// coding.cuh -- the experts' activation and the block-128 e4m3 coding of fp32
// values, as the dispatch codes its rows: scale = amax / 448 (fp32 division), code = e4m3 round to
// nearest even of v / scale (fp32 division), saturating; a block of zeros has
// scale 0 and zero bytes.  A NaN makes its block's scale and codes NaN (the
// dispatch leaves NaN out of amax, so a block of nothing but NaN is coded as
// zeros there; a norm or a product should not lose it).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

// silu(g) * u with the fast exponential and division (about (|g| + 4) 2^-23 of
// the result off; the sums g and u come with more).  For g below -87 the
// quotient is 0 where the formula has a value of magnitude 2^-119 or less.
__device__ __forceinline__ float silu_mul(float g, float u) {
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// |v| as bits: their order as unsigned integers is that of the magnitudes,
// with NaN above infinity, so an integer maximum finds amax and keeps NaN.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    return m;
}

__device__ __forceinline__ float block_scale(uint32_t amax) {
    return __fdiv_rn(__uint_as_float(amax), 448.0f);
}

// Four values to four codes, the first in the low byte.
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, float scale) {
    const uint32_t lo = (uint32_t)__nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(a, scale), __fdiv_rn(b, scale)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = (uint32_t)__nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(c, scale), __fdiv_rn(d, scale)), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Four values times the reciprocal of the scale: a rounding more than the
// division, which moves a code only where the quotient is within an ulp of the
// middle of two codes; a fraction of the division's instructions.
__device__ __forceinline__ uint32_t code4_by(float a, float b, float c, float d, float inv) {
    const uint32_t lo = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv),
                                                           __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv),
                                                           __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Below this scale a reciprocal may overflow: multiply values and scale by
// kTinyUp first.
constexpr float kTinyScale = 0x1p-120f, kTinyUp = 0x1p100f;

// The factor that takes a block's values to codes and, where the scale is tiny,
// what to multiply the values by before it (else 1).  A block with scale 0 has
// zero bytes, not these products' (negative zeros have a code of their own).
__device__ __forceinline__ float code_factor(float scale, float *first) {
    *first = scale < kTinyScale ? kTinyUp : 1.0f;
    return scale == 0.0f ? 0.0f : __frcp_rn(scale * *first);
}

// Eight values of a block whose scale is known.
__device__ __forceinline__ uint2 code8_by(float (&v)[8], float scale) {
    float first;
    const float inv = code_factor(scale, &first);
    if (first != 1.0f)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = scale == 0.0f ? 0.0f : v[i] * first;
    return make_uint2(code4_by(v[0], v[1], v[2], v[3], inv), code4_by(v[4], v[5], v[6], v[7], inv));
}

}  // namespace moe
