// topk.cu -- moe_topk: a router's choice of experts and their weights from logits.
//
// What chooses is turned into 32-bit integers whose order is the values', so that the
// choice is integer maxima.  Without a bias the integers are the logits themselves,
// exactly.  With one, c = s + bias comes from fp32; where two neighbours among the
// first R + 1, or the kept runs' worths and the others', are closer than both their
// errors, the token's candidates are evaluated and ordered again more exactly (one
// token in 2000 at 256 experts).  A warp has a token, or, for up to eight of up to 512
// experts, four.
//
// Measured: 32767 tokens, 8 of 128 experts 11.6 us (1.6 TB/s), of 256 16.7 (2.1 TB/s), with
// a bias and four of eight runs kept 37.5; 2048 tokens, 8 of 256 4.3, with a bias 7.0, and
// four of eight runs kept 8.5, 32 of 1024 24.  It is bound
// by instructions: at 128 experts about 150 a token and lane of eight, most of them in
// the sorting networks (19 exchanges for eight keys, 12 for each further eight and each
// doubling of the lanes); one token after another by whole warps took 26 us.  Few
// tokens are one chain of loads, exchanges and exponentials.
#include <cmath>

#include "check.h"
#include "common.cuh"
#include "launch.h"
#include "trace.h"

namespace moe {

struct Router {
    int rows, E, R, score, groups, kept, best, renorm, per;
    unsigned per_inv;  // floor(e / per) == (e * per_inv) >> 20 for e < 1024
    uint32_t ends;     // bit q: expert 32 q + 31 is the last of its run
    float scale;
    const float *logits, *bias;
    int32_t *idx;
    float *w;
};

// Order-preserving integers of floats: larger for larger, the two zeros alike;
// kLowest for -infinity and NaN.  0 is left for "not there".
constexpr uint32_t kLowest = 0x007fffffu;
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return v == v ? k : kLowest;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// A score as it is compared, with the fast exponential, e^x within (2 + 1.16 |x|) 2^-23
// of itself, and the fast quotient, within 2^-22.
__device__ __forceinline__ float score_about(int score, float l, float top, float inv_sum) {
    return score == MOE_SCORE_SIGMOID ? __fdividef(1.0f, 1.0f + __expf(-l))
                                      : __expf(l - top) * inv_sum;
}

// The same of several logits: which score it is, is asked once, and no one waits for
// another's (32 a lane by themselves, each behind its own branches, took 3 us).
template <int n>
__device__ __forceinline__ void scores_about(int score, const float (&l)[n], float top,
                                             float inv_sum, float (&s)[n]) {
    if (score == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < n; ++i) s[i] = score_about(MOE_SCORE_SIGMOID, l[i], 0.0f, 0.0f);
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) s[i] = score_about(MOE_SCORE_SOFTMAX, l[i], top, inv_sum);
    }
}

// How far c is then from the 64-bit one, by its magnitude.  A sigmoid: s (1 - s) of the
// exponential's error, at most 0.56 * 2^-23, the addition's 2^-24 and the quotient's
// 2^-22, less than 2^-21 together.  A softmax: at most 2.5 * 2^-23 by the exponential,
// its argument's rounding less than 2^-24, and the sum of up to 1024 exponentials, of
// which no more than 32 are added one after another, within 50 * 2^-24: less than
// 2^-18.  The addition of the bias rounds once.
__device__ __forceinline__ float error_of(int score, float c) {
    return (score == MOE_SCORE_SIGMOID ? 0x1p-21f : 0x1p-18f) + fabsf(c) * 0x1p-23f;
}

// A run's worth by its two largest values is compared by its half: the sum itself may be
// past fp32 where the biases are not.  worth_slack: the errors of two runs' worths
// together, by the values of one (half of each value's twice; or its first value's twice).
__device__ __forceinline__ float half_sum(float a, float b) { return 0.5f * a + 0.5f * b; }
__device__ __forceinline__ float worth_slack(int score, bool sums, float a, float b) {
    return error_of(score, a) + error_of(score, sums ? b : a);
}

// The same score with the accurate ones, for the weights.
__device__ __forceinline__ float score32(int score, float l, float top, float inv_sum) {
    return score == MOE_SCORE_SIGMOID ? 1.0f / (1.0f + expf(-l)) : expf(l - top) * inv_sum;
}

// The run of expert e, of E or of the padding behind them.
__device__ __forceinline__ int run_of(const Router &p, int e) {
    return min((int)((e * p.per_inv) >> 20), 31);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// Experts a lane holds, and the tokens of a CTA by it: shared memory bounds them.
__host__ __device__ constexpr int topk_warps(int C) { return C <= 16 ? 4 : 2; }

// ------------------------------------------------------------ nearer than fp32
//
// What fp32 cannot order is evaluated again, in fixed point with 2^-46 as the unit from
// pairs of fp32 numbers (sigmoid scores; 17 units off at most), and in fp64 where that
// is not enough either, or not at hand.  The GPU has few fp64 units: a token's
// candidates take them 4 us, the other way 1.

// A warp's room for it.
template <int C>
struct Exact {
    long long c[C * 32];  // or doubles
    uint16_t list[C * 32];
};

__device__ __forceinline__ void two_sum(float &a, float &b) {  // a + b, and what it lost
    const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
    b = __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t));
    a = s;
}

// 2^(j / 16) as pairs.
__constant__ float kRootHigh[16] = {
    0x1p+0f,        0x1.0b5586p+0f, 0x1.172b84p+0f, 0x1.2387a6p+0f, 0x1.306fep+0f,  0x1.3dea64p+0f,
    0x1.4bfdaep+0f, 0x1.5ab07ep+0f, 0x1.6a09e6p+0f, 0x1.7a1148p+0f, 0x1.8ace54p+0f, 0x1.9c4918p+0f,
    0x1.ae89fap+0f, 0x1.c199bep+0f, 0x1.d5818ep+0f, 0x1.ea4afap+0f};
__constant__ float kRootLow[16] = {
    0.0f,             0x1.9f3122p-25f, -0x1.c15742p-27f, 0x1.ceac48p-25f,
    0x1.4636e2p-25f,  0x1.824684p-25f, -0x1.593abcp-25f, -0x1.5bd5ecp-27f,
    0x1.9fcef4p-26f,  -0x1.829fdp-25f, 0x1.15506ep-27f,  0x1.51f848p-27f,
    -0x1.a94b14p-26f, -0x1.3d56b2p-27f, -0x1.822dbcp-27f, 0x1.52486cp-27f};

// 1 / (1 + exp(-l)) in units of 2^-46.  exp(y) = 2^(n / 16) e^r with |r| <= ln 2 / 32:
// y - n ln 2 / 16 with that constant in three parts, of which n times the first two are
// exact; e^r by its series; the sum and the quotient with their remainders.  Beyond 60
// it is 0 or 1 as far as a unit goes.
__device__ __forceinline__ long long sigmoid_fixed(float l) {
    const float y = -fminf(fmaxf(l, -60.0f), 60.0f);
    const float n = rintf(__fmul_rn(y, 23.083120654223414f));
    float h = __fmaf_rn(-n, 0x1.62ep-5f, y), e = -__fmul_rn(n, 0x1.0bep-19f);
    two_sum(h, e);
    e = __fmaf_rn(-n, 0x1.be8e7cp-31f, e);
    two_sum(h, e);  // r
    const float p = __fmul_rn(h, h), pe = __fmaf_rn(h, h, -p);
    const float cube = __fmul_rn(
        __fmul_rn(h, p),
        __fmaf_rn(h, __fmaf_rn(h, __fmaf_rn(h, 1.0f / 720, 1.0f / 120), 1.0f / 24), 1.0f / 6));
    float low = __fadd_rn(__fmaf_rn(0.5f, pe, cube), __fmaf_rn(e, h, e));
    float one = 1.0f, r = h, half = __fmul_rn(0.5f, p);
    two_sum(one, r);
    two_sum(one, half);  // e^r = one + low
    low = __fadd_rn(__fadd_rn(r, half), low);
    const int k = (int)n, j = k & 15;
    const float th = kRootHigh[j], by = __int_as_float(((k >> 4) + 127) << 23);
    float eh = __fmul_rn(one, th);
    float el = __fadd_rn(__fmaf_rn(one, th, -eh), __fmaf_rn(one, kRootLow[j], __fmul_rn(low, th)));
    eh = __fmul_rn(eh, by);
    el = __fmul_rn(el, by);
    float d = 1.0f;
    two_sum(d, eh);
    eh = __fadd_rn(eh, el);
    two_sum(d, eh);  // the denominator, d + eh
    const float q = __fdiv_rn(1.0f, d);
    const float rest = __fmul_rn(q, __fmaf_rn(-q, eh, __fmaf_rn(-q, d, 1.0f)));
    return __float2ll_rn(q * 0x1p46f) + __float2ll_rn(rest * 0x1p46f);
}
// Two values of one or two scores each that are so near are not told apart by it.
constexpr long long kNear = 128, kNone = -(1LL << 62);

// An expert's c (its score without a bias), in either way; a masked one's is lowest.
template <class T>
__device__ __forceinline__ T value_exact(const Router &p, const float *l, int e, float top,
                                         double sum) {
    const float v = l[e], b = p.bias ? p.bias[e] : 0.0f;
    if constexpr (T(0.5) == T(0)) {
        if (v == -INFINITY || !(fabsf(b) < 16384.0f) || v != v) return kNone;
        return sigmoid_fixed(v) + __float2ll_rn(b * 0x1p46f);
    } else {
        double c = p.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-(double)v))
                                                : exp((double)v - (double)top) / sum;
        c += (double)b;
        return v != -INFINITY && c == c ? c : -(double)INFINITY;
    }
}
// Whether fixed point holds the bias, and the difference of two runs' worths (-infinity
// and NaN are as good as a masked logit).
__device__ __forceinline__ bool fits(float b) {
    return fabsf(b) < 16384.0f || b != b || b == -INFINITY;
}

__device__ __forceinline__ double sum64(const Router &p, const float *l, float top) {
    if (p.score == MOE_SCORE_SIGMOID) return 1.0;
    double sum = 0.0;
    for (int e = threadIdx.x & 31; e < p.E; e += 32) sum += exp((double)l[e] - (double)top);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    return sum;
}

// The kept runs, one bit each, by all lanes of a warp.  False: not told apart.
template <class T>
__device__ __noinline__ bool kept_exact(const Router &p, const float *l, long long *room, float top,
                                        uint32_t *kept) {
    constexpr bool kFixed = T(0.5) == T(0);
    T *c = reinterpret_cast<T *>(room);
    const int lane = threadIdx.x & 31;
    const double sum = kFixed ? 1.0 : sum64(p, l, top);
    bool ok = true;
    for (int e = lane; e < p.E; e += 32) {
        c[e] = value_exact<T>(p, l, e, top, sum);
        if (kFixed && p.bias) ok &= fits(p.bias[e]);
    }
    __syncwarp();
    const T none = kFixed ? T(kNone) : T(-(double)INFINITY);
    T worth = none;
    if (lane < p.groups) {
        T a = none, b = none;  // the two largest
        for (int e = lane * p.per; e < (lane + 1) * p.per; ++e) {
            const T x = c[e];
            b = max(b, min(a, x));
            a = max(a, x);
        }
        worth = p.best == 1 ? a : b == none ? none : a + b;
    }
    int before = 0;
    bool near = false;
    for (int g = 0; g < p.groups; ++g) {
        const T o = __shfl_sync(kFull, worth, g);
        before += o > worth || (o == worth && g < lane);
        if (kFixed && g != lane && worth != none && o != none)
            near |= o - worth <= T(kNear) && worth - o <= T(kNear);
    }
    __syncwarp();
    *kept = __ballot_sync(kFull, lane < p.groups && before < p.kept);
    return __all_sync(kFull, ok && !(near && lane < p.groups));
}

// The choice, by all lanes of a warp, of the kept experts whose c is `least` or more in
// fp32, in 64 bits: lane r gets the r-th.  Only with a bias.
__device__ __noinline__ void choose64(const Router &p, const float *l, long long *room,
                                      uint16_t *list, float top, uint32_t kept, float least,
                                      int *mine) {
    double *c = reinterpret_cast<double *>(room);
    const int lane = threadIdx.x & 31;
    const double sum = sum64(p, l, top);
    int n = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {  // listed in the order of their index
        const int e = e0 + lane;
        bool in = e < p.E && (kept >> run_of(p, e) & 1u);
        if (in) {
            const float v = l[e];
            float x = score_about(p.score, v, top, (float)(1.0 / sum)) + p.bias[e];
            if (v == -INFINITY || x != x) x = -INFINITY;
            in = x >= least;
        }
        const unsigned who = __ballot_sync(kFull, in);
        if (in) list[n + __popc(who & ((1u << lane) - 1u))] = (uint16_t)e;
        n += __popc(who);
    }
    __syncwarp();
    for (int j = lane; j < n; j += 32) c[j] = value_exact<double>(p, l, list[j], top, sum);
    __syncwarp();
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        int before = 32;
        if (j < n) {
            before = 0;
            for (int o = 0; o < n; ++o) before += c[o] > c[j] || (c[o] == c[j] && o < j);
        }
        for (int o = 0; o < 32; ++o)  // candidate j0 + o goes to the lane of its rank
            if (__shfl_sync(kFull, before, o) == lane) *mine = list[j0 + o];
    }
    __syncwarp();
}

// A lane's logits or biases: v[4 q + j] is expert 128 q + 4 lane + j; `none` behind the
// last.  By plain loads: the kernel before may write them while this one waits for it.
__device__ __forceinline__ int expert_at(int i) {
    return (i >> 2) * 128 + (threadIdx.x & 31) * 4 + (i & 3);
}
template <int C>
__device__ __forceinline__ void load_row(const Router &p, const float *l, float none,
                                         float (&v)[C]) {
    const bool quads = (p.E & 3) == 0;  // then every row starts on 16 bytes
#pragma unroll
    for (int q = 0; q < C / 4; ++q) {
        const int e = expert_at(4 * q);
        float4 f = make_float4(none, none, none, none);
        if (quads) {
            if (e < p.E) f = *reinterpret_cast<const float4 *>(l + e);
        } else {
            if (e < p.E) f.x = l[e];
            if (e + 1 < p.E) f.y = l[e + 1];
            if (e + 2 < p.E) f.z = l[e + 2];
            if (e + 3 < p.E) f.w = l[e + 3];
        }
        v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
    }
}

// What is compared, c or the logits: masked experts last, those behind the last and
// those of runs that are not kept not there at all.
template <int C>
__device__ __forceinline__ void make_keys(const Router &p, const float (&v)[C],
                                          const float (&b)[C], float top, float inv_sum,
                                          uint32_t kept, uint32_t (&key)[C]) {
    if (p.bias) {
        float c[C];
        scores_about(p.score, v, top, inv_sum, c);
#pragma unroll
        for (int i = 0; i < C; ++i) key[i] = key_of(v[i] == -INFINITY ? v[i] : c[i] + b[i]);
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) key[i] = key_of(v[i]);
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (expert_at(i) >= p.E) key[i] = 0u;
    if (kept != ~0u) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (!(kept >> run_of(p, expert_at(i)) & 1u)) key[i] = 0u;
    }
}

// What a run's worth is made of: c, or the scores where there is no bias and two are
// added.
template <int n>
__device__ __forceinline__ void run_values(const Router &p, const float (&v)[n],
                                           const uint32_t (&key)[n], float top, float inv_sum,
                                           bool scored, float (&c)[n]) {
    if (scored)
        scores_about(p.score, v, top, inv_sum, c);
    else
#pragma unroll
        for (int i = 0; i < n; ++i) c[i] = value_of(key[i]);
#pragma unroll
    for (int i = 0; i < n; ++i)
        if (key[i] <= kLowest) c[i] = -INFINITY;
}

// The runs that are kept, one bit each; keys are of all experts.
template <int C>
__device__ __forceinline__ uint32_t kept_runs(const Router &p, const float *l, const float (&v)[C],
                                              const uint32_t (&key)[C], float top, float inv_sum,
                                              long long *room) {
    const int lane = threadIdx.x & 31;
    float slack = 0.0f;  // of two runs' worths
    uint32_t mine = 0;   // lane g: the worth of run g
    const bool sums = p.best == 2, scored = !p.bias && sums;
    if (p.per >= 4 && p.per <= 128 && (p.per & (p.per - 1)) == 0) {
        // a run is p.per / 4 neighbouring lanes' quads: their best two by exchanges.  The
        // way below asks all lanes for each run: 2048 tokens, 256 experts in eight runs
        // 24.0 us that way, 8.5 this
        float worths[C];
        run_values(p, v, key, top, inv_sum, scored, worths);
#pragma unroll
        for (int q = 0; q < C / 4; ++q) {
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int i = 4 * q; i < 4 * q + 4; ++i) {
                b = fmaxf(b, fminf(a, worths[i]));
                a = fmaxf(a, worths[i]);
            }
            for (int d = p.per >> 3; d > 0; d >>= 1) {
                const float oa = __shfl_xor_sync(kFull, a, d), ob = __shfl_xor_sync(kFull, b, d);
                b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                a = fmaxf(a, oa);
            }
            const float worth = sums ? half_sum(a, b) : a;
            if (worth > -INFINITY) slack = fmaxf(slack, worth_slack(p.score, sums, a, b));
            // to lane g from the first lane of run g
            const int e = lane * p.per;
            const float got = __shfl_sync(kFull, worth, (e & 127) >> 2);
            if (lane < p.groups && (e >> 7) == q) mine = key_of(got);
        }
        slack = warp_max(slack);
    } else {
        for (int g = 0; g < p.groups; ++g) {
            uint32_t a = 0, b = 0;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (run_of(p, expert_at(i)) != g) continue;
                uint32_t k = key[i];
                if (scored && k > kLowest) k = key_of(score_about(p.score, v[i], top, inv_sum));
                b = max(b, min(a, k));
                a = max(a, k);
            }
            const uint32_t first = __reduce_max_sync(kFull, a);
            uint32_t worth = first, second = first;
            if (sums) {
                const unsigned who = __ballot_sync(kFull, a == first);
                // the second largest: the others' first, or this lane's second
                const uint32_t rest = (who & (who - 1)) || a != first ? a : b;
                second = __reduce_max_sync(kFull, rest);
                worth = key_of(half_sum(value_of(first), value_of(second)));
            }
            if (worth > kLowest)
                slack = fmaxf(slack,
                              worth_slack(p.score, sums, value_of(first), value_of(second)));
            if (lane == g) mine = worth;
        }
    }
    int before = 0;
    for (int g = 0; g < p.groups; ++g) {
        const uint32_t o = __shfl_sync(kFull, mine, g);
        before += o > mine || (o == mine && g < lane);
    }
    const bool run = lane < p.groups;
    uint32_t kept = __ballot_sync(kFull, run && before < p.kept);
    if (p.bias || sums) {
        // the least kept and the best of the others
        const uint32_t in = __reduce_min_sync(kFull, run && before < p.kept ? mine : ~0u);
        const uint32_t out = __reduce_max_sync(kFull, run && before >= p.kept ? mine : 0u);
        if (out > kLowest && value_of(in) - value_of(out) <= slack)
            if (p.score != MOE_SCORE_SIGMOID || !kept_exact<long long>(p, l, room, top, &kept))
                kept_exact<double>(p, l, room, top, &kept);
    }
    return kept;
}

// The R largest keys, one after another, equal ones by their index: lane r gets the
// r-th's expert.  With a bias those behind the R-th too that may be before it as far as
// fp32 knows, n in all, `over` where they are more than the lanes; `least` is as far as
// they go.
struct Chosen {
    int mine, n;
    float c, least;  // what chose it
    bool over;
};

template <int C>
__device__ __forceinline__ Chosen take_any(const Router &p, uint32_t (&key)[C]) {
    const int lane = threadIdx.x & 31;
    Chosen got = {0, 0, -INFINITY, -INFINITY, false};
    for (int r = 0;; ++r) {
        if (r == p.R && !p.bias) break;
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < C; ++i) m = max(m, key[i]);
        const uint32_t most = __reduce_max_sync(kFull, m);
        if (most == 0u) break;  // no one is left
        const float c = value_of(most);
        // a masked one is behind all others, by its index
        if (r >= p.R && (!(c >= got.least) || c == -INFINITY)) break;
        got.over = r == 32;
        if (got.over) break;
        if (r == p.R - 1) got.least = c > -INFINITY ? c - 2.0f * error_of(p.score, c) : -INFINITY;
        // its place in the lanes that have it, and of those the lowest
        int i0 = 0;
#pragma unroll
        for (int i = C - 1; i >= 0; --i)
            if (key[i] == most) i0 = i;
        const unsigned at = m == most ? (unsigned)expert_at(i0) : ~0u;
        const unsigned first = __reduce_min_sync(kFull, at);
        if (at == first) {
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (i == i0) key[i] = 0u;
        }
        if (lane == r) got.mine = (int)first, got.c = c;
        got.n = r + 1;
    }
    return got;
}

// The candidates of take_any in the order of their exact values, in fixed point.  Short,
// and by the lanes that have them: it is code that one token in 2000 needs, which comes
// from beyond the caches for it.  False: not told apart.
__device__ __forceinline__ bool order_fixed(const Router &p, const float *l, uint16_t *list,
                                            Chosen &got) {
    const int lane = threadIdx.x & 31;
    const bool in = lane < got.n;
    const long long c = in ? value_exact<long long>(p, l, got.mine, 0.0f, 1.0) : kNone;
    bool ok = !got.over && (!in || fits(p.bias[got.mine]));
    int before = 0;
    for (int o = 0; o < got.n; ++o) {
        const long long y = __shfl_sync(kFull, c, o);
        before += y > c || (y == c && o < lane);
        if (o != lane && c != kNone && y != kNone) ok &= y - c > kNear || c - y > kNear;
    }
    if (in) list[before] = (uint16_t)got.mine;
    __syncwarp();
    if (in) got.mine = list[lane];
    __syncwarp();
    return __all_sync(kFull, ok);
}

__device__ __forceinline__ bool near(const Router &p, uint32_t last, uint32_t next) {
    const float a = value_of(last), b = value_of(next);
    // (two of +infinity, whose difference is NaN, too)
    return b > -INFINITY && !(a - b > error_of(p.score, a) + error_of(p.score, b));
}

// One token, by all lanes of a warp.
template <int C>
__device__ __noinline__ void token_by_warp_apart(const Router &p, int row, Exact<C> &exact);
template <int C>
__device__ __forceinline__ void token_by_warp(const Router &p, int row, Exact<C> &exact) {
    const int lane = threadIdx.x & 31;
    const float *l = p.logits + (size_t)row * p.E;
    float v[C], b[C] = {};
    load_row(p, l, -INFINITY, v);
    if (p.bias) load_row(p, p.bias, 0.0f, b);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < C; ++i)
        bad |= v[i] != v[i] || (p.score == MOE_SCORE_SOFTMAX && v[i] == INFINITY);
    bad = __any_sync(kFull, bad);
    // the softmax's maximum and sum, where a value needs them
    const bool scores = p.bias || (p.groups > p.kept && p.best == 2);
    float top = 0.0f, inv_sum = 1.0f;
    if (p.score == MOE_SCORE_SOFTMAX && (scores || !p.renorm)) {
        top = v[0];
#pragma unroll
        for (int i = 1; i < C; ++i) top = fmaxf(top, v[i]);
        top = warp_max(top);
        float sum = 0.0f;
        if (top > -INFINITY)
#pragma unroll
            for (int i = 0; i < C; ++i) sum += expf(v[i] - top);
        sum = warp_sum(sum);
        inv_sum = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    uint32_t key[C], kept = ~0u;
    make_keys(p, v, b, top, inv_sum, ~0u, key);
    if (p.groups > p.kept) {
        kept = kept_runs(p, l, v, key, top, inv_sum, exact.c);
        if ((p.per & 3) == 0) {  // a quad is of one run
#pragma unroll
            for (int q = 0; q < C / 4; ++q)
                if (!(kept >> run_of(p, expert_at(4 * q)) & 1u))
                    key[4 * q] = key[4 * q + 1] = key[4 * q + 2] = key[4 * q + 3] = 0u;
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (!(kept >> run_of(p, expert_at(i)) & 1u)) key[i] = 0u;
        }
    }
    Chosen got = take_any(p, key);
    // (a softmax that is no number has nothing to be ordered by more exactly: all of its
    // exact values are NaN)
    if (p.bias && !(bad && p.score == MOE_SCORE_SOFTMAX)) {
        // neighbours that are nearer than their errors, or some that may be before the R-th
        const float next = __shfl_down_sync(kFull, got.c, 1);
        const bool close = lane + 1 < got.n && next > -INFINITY &&
                           got.c - next <= error_of(p.score, got.c) + error_of(p.score, next);
        if (__any_sync(kFull, close) || got.over || got.n > p.R)
            if (p.score != MOE_SCORE_SIGMOID || !order_fixed(p, l, exact.list, got)) {
                int mine = 0;
                choose64(p, l, exact.c, exact.list, top, kept, got.least, &mine);
                got.mine = mine;
            }
    }
    // the weights, lane r the r-th; sums over as many lanes as there may be
    const int half = p.R > 8 ? 16 : 4;
    const bool chosen = lane < p.R;
    float lv = chosen ? l[got.mine] : -INFINITY;
    if (p.bias) {  // one that its bias takes out of service is as good as masked
        const float b = chosen ? p.bias[got.mine] : 0.0f;
        if (!(b > -INFINITY)) lv = -INFINITY;
    }
    float s = 0.0f;
    if (p.renorm) {
        // all of them times exp(-m), so that small ones keep their ratios
        float m = lv;
        for (int d = half; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
        if (lv > -INFINITY)
            s = p.score == MOE_SCORE_SOFTMAX ? expf(lv - m)
                : m >= 0.0f                  ? score32(p.score, lv, top, inv_sum)
                                             : expf(lv - m) / (1.0f + expf(lv));
        float sum = s;
        for (int d = half; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
        s = sum > 0.0f ? s / sum : 0.0f;
    } else if (lv > -INFINITY) {
        s = score32(p.score, lv, top, inv_sum);
    }
    if (chosen) {
        p.idx[(size_t)row * p.R + lane] = got.mine;
        p.w[(size_t)row * p.R + lane] = bad ? __uint_as_float(0x7fffffffu) : s * p.scale;
    }
}

// (us with the compiler's own choice of registers, which spills, and with these: 2048 tokens,
// 8 of 384 with a bias 8.0 and 7.2, 8 of 256 with a bias and runs 9.8 and 8.5)
template <int C>
__global__ void __launch_bounds__(32 * topk_warps(C), C <= 8 ? 8 : 5) k_topk(const __grid_constant__ Router p) {
    constexpr int kWarps = topk_warps(C);
    __shared__ Exact<C> exact[kWarps];
    const int warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row = blockIdx.x * kWarps + warp;
    if (row < p.rows) token_by_warp(p, row, exact[warp]);
}

template <int C>
__device__ __noinline__ void token_by_warp_apart(const Router &p, int row, Exact<C> &exact) {
    token_by_warp(p, row, exact);
}

// ------------------------------------------------------------ eight lanes a token
//
// Up to eight experts of up to 512, four tokens a warp: lane `sub` of a token's eight
// holds experts 32 q + 4 sub .. + 3.  The eight largest keys come from sorting networks
// on the keys alone (two instructions an exchange), eight at a time in a lane and then
// over the lanes; a key's place is how many of them are larger.  Where keys are equal
// or too near each other, or runs' worths are, the token goes through the warp's way
// above, all lanes together.

constexpr int kFastMost = 8, kFastWarps = 4;

__device__ __forceinline__ void exchange(uint32_t &a, uint32_t &b) {  // the larger to a
    const uint32_t m = max(a, b);
    b = min(a, b);
    a = m;
}
// Batcher's odd-even merge sort of eight, largest first.
__device__ __forceinline__ void sort8(uint32_t (&k)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) exchange(k[i], k[i + 1]);
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        exchange(k[i], k[i + 2]);
        exchange(k[i + 1], k[i + 3]);
        exchange(k[i + 1], k[i + 2]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) exchange(k[i], k[i + 4]);
    exchange(k[2], k[4]);
    exchange(k[3], k[5]);
#pragma unroll
    for (int i = 1; i < 7; i += 2) exchange(k[i], k[i + 1]);
}
// The eight largest of a first and then a falling row, sorted again.
__device__ __forceinline__ void resort8(uint32_t (&k)[8]) {
#pragma unroll
    for (int d = 4; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) exchange(k[i], k[i + d]);
}

// S: experts a lane holds.
template <int S>
__global__ void __launch_bounds__(32 * kFastWarps, S <= 16 ? 8 : S <= 32 ? 6 : 3)
    k_topk_fast(const __grid_constant__ Router p) {
    constexpr int Q = S / 4, C = S <= 16 ? 4 : S <= 32 ? 8 : 16;
    // keys to look up by number, and later the room of the other way
    union Room {
        Exact<C> exact;
        uint32_t key[S][32];
    };
    __shared__ Room room[kFastWarps];
    __shared__ int chosen[kFastWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row0 = (blockIdx.x * kFastWarps + warp) * 4;
    if (row0 >= p.rows) return;
    const int row = row0 + (lane >> 3);
    const bool there = row < p.rows;
    const float *l = p.logits + (size_t)(there ? row : row0) * p.E;
    float v[S];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (32 * q + 4 * sub < p.E) f = *reinterpret_cast<const float4 *>(l + 32 * q + 4 * sub);
        v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
    }
    const auto over = [&](auto f, float x) {  // of the token's lanes
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) x = f(x, __shfl_xor_sync(kFull, x, d));
        return x;
    };
    const auto greater = [](float a, float b) { return fmaxf(a, b); };
    const auto less = [](float a, float b) { return fminf(a, b); };
    const auto plus = [](float a, float b) { return a + b; };
    // tokens whose logits are not numbers, too, go the other way
    bool slow = false;
#pragma unroll
    for (int i = 0; i < S; ++i) slow |= !(v[i] < INFINITY);
    const bool grouped = p.groups > p.kept, sums = p.best == 2;
    const bool scored = grouped && sums && !p.bias;
    float top = 0.0f, inv_sum = 1.0f;
    if (p.score == MOE_SCORE_SOFTMAX && (p.bias || scored || !p.renorm)) {
        top = v[0];
#pragma unroll
        for (int i = 1; i < S; ++i) top = fmaxf(top, v[i]);
        top = over(greater, top);
        float sum[4] = {};
        if (top > -INFINITY)
#pragma unroll
            for (int i = 0; i < S; ++i) sum[i & 3] += expf(v[i] - top);
        sum[0] = over(plus, (sum[0] + sum[1]) + (sum[2] + sum[3]));
        inv_sum = sum[0] > 0.0f ? 1.0f / sum[0] : 0.0f;
    }
    uint32_t key[S];
    if (p.bias) {
        float c[S];
        scores_about(p.score, v, top, inv_sum, c);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int e = 32 * q + 4 * sub;
            float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (e < p.E) b = *reinterpret_cast<const float4 *>(p.bias + e);
            c[4 * q] += b.x, c[4 * q + 1] += b.y, c[4 * q + 2] += b.z, c[4 * q + 3] += b.w;
        }
#pragma unroll
        for (int i = 0; i < S; ++i) key[i] = key_of(v[i] == -INFINITY ? v[i] : c[i]);
    } else {
#pragma unroll
        for (int i = 0; i < S; ++i) key[i] = key_of(v[i]);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)  // E is a multiple of four
        if (32 * q + 4 * sub >= p.E)
            key[4 * q] = key[4 * q + 1] = key[4 * q + 2] = key[4 * q + 3] = 0u;
    if (grouped) {
        // p.per is a multiple of 32: a run is p.per / 32 whole q, which all lanes share.
        // worth[q]: of the run that ends with q, else nothing
        float worth[Q], a = -INFINITY, b = -INFINITY, slack = 0.0f, worths[S];
        run_values(p, v, key, top, inv_sum, scored, worths);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float a0 = -INFINITY, b0 = -INFINITY;
#pragma unroll
            for (int i = 4 * q; i < 4 * q + 4; ++i) {
                b0 = fmaxf(b0, fminf(a0, worths[i]));
                a0 = fmaxf(a0, worths[i]);
            }
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) {
                const float oa = __shfl_xor_sync(kFull, a0, d), ob = __shfl_xor_sync(kFull, b0, d);
                b0 = fmaxf(fminf(a0, oa), fmaxf(b0, ob));
                a0 = fmaxf(a0, oa);
            }
            const bool starts = q == 0 || (p.ends >> (q - 1) & 1u), ends = p.ends >> q & 1u;
            b = starts ? b0 : fmaxf(fminf(a, a0), fmaxf(b, b0));
            a = starts ? a0 : fmaxf(a, a0);
            worth[q] = ends ? (sums ? half_sum(a, b) : a) : -INFINITY;
            if (worth[q] > -INFINITY) slack = fmaxf(slack, worth_slack(p.score, sums, a, b));
        }
        // lane sub ranks the runs that end with q = sub, sub + 8
        uint32_t ends = 0;
        float least = INFINITY, best = -INFINITY;
#pragma unroll
        for (int h = 0; h < (Q + 7) / 8; ++h) {
            float mine = -INFINITY;
#pragma unroll
            for (int q = 8 * h; q < 8 * h + 8; ++q)
                if (q < Q && q - 8 * h == sub) mine = worth[q < Q ? q : 0];
            int before = 0;
#pragma unroll
            for (int q = 0; q < Q; ++q)
                before += worth[q] > mine || (worth[q] == mine && q < 8 * h + sub);
            // a run without any expert in service may be among the kept: the other way
            const bool run = mine > -INFINITY, in = run && before < p.kept;
            ends |= (__ballot_sync(kFull, in) >> (lane & 24) & 0xffu) << (8 * h);
            if (in) least = fminf(least, mine);
            if (run && !in) best = fmaxf(best, mine);
        }
        least = over(less, least);
        best = over(greater, best);
        slow |= __popc(ends) != p.kept;
        slow |= best > -INFINITY && least - best <= (p.bias || sums ? slack : 0.0f);
        bool in = false;
#pragma unroll
        for (int q = Q - 1; q >= 0; --q) {
            if (p.ends >> q & 1u) in = ends >> q & 1u;
            if (!in) key[4 * q] = key[4 * q + 1] = key[4 * q + 2] = key[4 * q + 3] = 0u;
        }
    }
    // the eight largest keys, in order, in every lane of the token
    uint32_t t[8];
#pragma unroll
    for (int g = 0; g < S / 8; ++g) {
        uint32_t k[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = key[8 * g + i];
        sort8(k);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = g == 0 ? k[i] : max(t[i], k[7 - i]);
        if (g > 0) resort8(t);
    }
#pragma unroll
    for (int d = 1; d < 8; d *= 2) {
        uint32_t k[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = __shfl_xor_sync(kFull, t[7 - i], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = max(t[i], k[i]);
        resort8(t);
    }
    uint32_t last = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i == p.R - 1) last = t[i];
        if (i > 0 && i < p.R) slow |= p.bias ? near(p, t[i - 1], t[i]) : t[i] == t[i - 1];
    }
    slow |= last <= kLowest;
    // the keys that are, or may be, among the first R
    const float c = value_of(last);
    const uint32_t least = p.bias && last > kLowest ? key_of(c - 2.0f * error_of(p.score, c)) : last;
    uint64_t hits = 0;
    int n = 0;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const bool hit = key[i] >= least;
        hits |= (uint64_t)hit << i;
        n += hit;
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) n += __shfl_xor_sync(kFull, n, d);
    slow |= n != p.R;
    const unsigned slows = __ballot_sync(kFull, slow && there);
    slow = slows >> (lane & 24) & 0xffu;
    int *mine = chosen[warp] + (lane & 24);
#pragma unroll
    for (int i = 0; i < S; ++i) room[warp].key[i][lane] = key[i];
    if (!slow) {
        while (hits) {  // each lane its own: what it wrote itself
            const int i = __ffsll((long long)hits) - 1, e = 32 * (i >> 2) + 4 * sub + (i & 3);
            hits &= hits - 1;
            const uint32_t k = room[warp].key[i][lane];
            int place = 0;
#pragma unroll
            for (int o = 0; o < 8; ++o) place += t[o] > k;
            mine[place & 7] = e;
        }
    }
    __syncwarp();
    if (!slow && there) {
        // the weights: the token's lanes are among themselves here
        const unsigned who = 0xffu << (lane & 24);
        const int e = sub < p.R ? mine[sub] : 0;
        const float lv = sub < p.R ? l[e] : -INFINITY;
        float s = 0.0f;
        if (p.renorm) {
            float m = lv;
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(who, m, d));
            if (sub < p.R)
                s = p.score == MOE_SCORE_SOFTMAX ? expf(lv - m)
                    : m >= 0.0f                  ? score32(p.score, lv, top, inv_sum)
                                                 : expf(lv - m) / (1.0f + expf(lv));
            float sum = s;
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) sum += __shfl_xor_sync(who, sum, d);
            s = s / sum;
        } else if (sub < p.R) {
            s = score32(p.score, lv, top, inv_sum);
        }
        if (sub < p.R) {
            p.idx[(size_t)row * p.R + sub] = e;
            p.w[(size_t)row * p.R + sub] = s * p.scale;
        }
    }
    __syncwarp();
#pragma unroll 1
    for (int k = 0; k < 4; ++k)
        if (slows >> (8 * k) & 0xffu) token_by_warp_apart(p, row0 + k, room[warp].exact);
}

template <class K>
static cudaError_t launch(K kern, int tokens, int warps, const Router &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(((long long)p.rows + tokens - 1) / tokens));
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

static cudaError_t launch_topk(const Router &p, cudaStream_t st) {
    // us with a warp and with eight lanes a token, 256 experts: one token 3.5 and 3.2, 2048
    // 6.4 and 4.3, 32767 36 and 17; with a bias and four of eight runs 8 tokens 4.4 and
    // 6.2, 2048 8.4 and 10.7, 8192 16 and 20.5, 12288 22.2 and 21.7, 16384 28 and 24.5,
    // 32767 52 and 37.5: there some tokens go the warp's way after the other
    if (p.R <= kFastMost && p.E >= 32 && p.E <= 512 && p.E % 4 == 0 &&
        (p.groups == p.kept || p.per % 32 == 0) && (!p.bias || p.rows > 96 * sm_count())) {
        const auto kern = p.E <= 128   ? k_topk_fast<16>
                          : p.E <= 256 ? k_topk_fast<32>
                          : p.E <= 384 ? k_topk_fast<48>
                                       : k_topk_fast<64>;
        return launch(kern, 4 * kFastWarps, kFastWarps, p, st);
    }
    const auto kern = p.E <= 128 ? k_topk<4> : p.E <= 256 ? k_topk<8> : p.E <= 512 ? k_topk<16> : k_topk<32>;
    const int warps = p.E <= 512 ? topk_warps(16) : topk_warps(32);
    return launch(kern, warps, warps, p, st);
}

}  // namespace moe

extern "C" int moe_topk(const moe_shape *sh, int score, int groups, int kept, int best, int renorm,
                        float scale, const float *logits, const float *bias, int32_t *topk_idx,
                        float *topk_w, void *stream) {
    MOE_TRACE_CALL();
    moe_sizes z;
    const int rc = moe_sizes_query(sh, &z);
    if (rc != MOE_OK) return rc;
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
    if (groups < 1 || sh->E % groups != 0 || kept < 1 || kept > groups || !std::isfinite(scale))
        return MOE_EINVAL;
    const int per = sh->E / groups;
    if (best < 1 || best > 2 || best > per || sh->R > kept * per) return MOE_EINVAL;
    if (groups > MOE_MAX_GROUPS) return MOE_ENOTSUP;
    const int64_t rows = (int64_t)sh->N * sh->T;
    if (!moe::ok_buffer(logits, rows * sh->E * 4) || !moe::ok_optional(bias) ||
        !moe::ok_buffer(topk_idx, z.bytes_topk_idx) || !moe::ok_buffer(topk_w, z.bytes_topk_idx))
        return MOE_EINVAL;
    if (rows == 0) return MOE_OK;
    if (rows >= ((int64_t)1 << 31) - 64) return MOE_ENOTSUP;
    const unsigned inv = ((1u << 20) + per - 1) / per;
    uint32_t ends = 0;
    for (int q = 0; q < 32 && 32 * q + 31 < sh->E; ++q)
        if ((32 * q + 32) % per == 0) ends |= 1u << q;
    const moe::Router p = {(int)rows, sh->E, sh->R, score, groups, kept, best,     renorm != 0,
                           per,       inv,   ends,  scale, logits, bias, topk_idx, topk_w};
    return moe::launch_topk(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                      : MOE_ECUDA;
}
