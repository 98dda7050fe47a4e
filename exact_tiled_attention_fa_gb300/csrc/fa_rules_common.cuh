// fa_rules_common.cuh -- what the kernels of attention under score rules share.
//
// Scores.  With x = scale q.k, a cap c > 0 makes it c tanh(x / c), whose slope is 1 - tanh^2; a bias then takes
// slope_h |i - j| off (i, j the positions of query and key).  In base 2, as the exponentials want them:
// mult * (tanh(cap_in * S) - slope * |i - j|), S = q.k, slope = slope_h * bias_in.
#pragma once

#include <cstdint>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"
#include "ptx.cuh"

namespace fa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

constexpr int kRulesItems = 4;  // records of work items on their way from a CTA's producer to its other roles

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The cap.  tanh(u) for |u| <= kWideRange is u P(u^2) with P the minimax polynomial for tanh(u) / u (Remez exchange on
// u^2): degree n = 2 up to kNearRange (relative error 1.2e-6), 3 up to kMidRange (1.1e-6), 5 up to kWideRange (5.9e-7).  With
// cap_in and mult in its coefficients a capped score is S Q(S^2): n + 1 operations and the one that takes the maximum
// off it anyway.  (What bounds them is the FMA units, 128 lanes an SM, whether two operations go in one instruction or not.
// Causal prefill of 4 sequences of 4097 tokens, 16 heads of 128, a cap of 50 that leaves most tiles in the near range: a
// polynomial of degree 5 for every argument, scaled before it, 487 us, the three 348 when they were chosen, 360 with what
// cap_range_seen adds, without a cap 286.)
// Other arguments take 1 - 2 / (1 + e^2u): two operations of the special function unit that the exponentials also need
// (586 us for all tiles one by one, 562 by pairs).  The form goes by the largest of a warp's scores in a tile, 32 x 128 of
// them (backward 32 x 64), so one score near the cap is dear: scores of deviation 10 at the same shape 456 us.
// The exponential form's absolute error of 2e-7 is one of 1e-5 of a weight at a cap of 50.  And a score beyond the cap is no
// reason for one far below it to be off by 2e-7 caps, 0.01 of a score of 5 at a cap of 1e5: above kFarCap, where that error
// is a hundredth of a weight's rounding to bf16, scores up to kNearRange take their polynomial beside it too.  (For every cap
// that costs 1.0 - 1.4 times the time of the tiles it is for.)
// +-infinity gives +-1, NaN NaN.  (The device's own tanh instruction is off by 2^-11 of its result: at a score of 20
// by 0.01, and the weight by as much.)
constexpr float kNearRange = 0.3f, kMidRange = 0.55f, kWideRange = 1.f;
constexpr float kFarCap = 128.f;
#define FA_TANH_NEAR 0.999998838848, -0.333100215997, 0.126339459894
#define FA_TANH_MID 0.999998880298, -0.333213872584, 0.131312313762, -0.0426959989808
#define FA_TANH_WIDE 0.999999413602, -0.333290423701, 0.132814338124, -0.051605672318, 0.0167431133877, -0.00306705973621

__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }

// Q of a pair of scores; a capped score is s * Q.
template <int N>
__device__ __forceinline__ float2 cap_factor(float2 s, const float2 (&c)[N])
{
    const float2 w = __fmul2_rn(s, s);
    float2 q = c[N - 1];
#pragma unroll
    for (int i = N - 2; i >= 0; --i) q = __ffma2_rn(w, q, c[i]);
    return q;
}

// tanh of k * s, of any size.
__device__ __forceinline__ float tanh_each(float s, float k)
{
    constexpr float c[] = {FA_TANH_NEAR};
    const float y = fmaf(-2.f, rcp_approx(1.f + ex2(s * (k * (2.f * kLog2e)))), 1.f);
    const float u = s * k, w = u * u;
    return fabsf(u) <= kNearRange ? u * fmaf(w, fmaf(w, c[2], c[1]), c[0]) : y;  // (NaN: y, which is NaN)
}

// tanh of N numbers k * s, in place, beyond the polynomials' ranges or, with `far`, of any size.
template <int N>
__device__ __forceinline__ void tanh_any(float* s, float k, bool far)
{
    if (!far) {
        const float2 k2 = two(k * (2.f * kLog2e));
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 z = __fmul2_rn(make_float2(s[i], s[i + 1]), k2);
            const float2 e = __fadd2_rn(make_float2(ex2(z.x), ex2(z.y)), two(1.f));
            const float2 y = __ffma2_rn(two(-2.f), make_float2(rcp_approx(e.x), rcp_approx(e.y)), two(1.f));
            s[i] = y.x;
            s[i + 1] = y.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = tanh_each(s[i], k);
    }
}

// Whether every lane's |S| (its largest, mx) lies in the polynomials' ranges: 3 the near one, 2 the middle one, 1 the wide
// one, 0 none.  kSettled stands for scores that are tanh already (tree_settle).
constexpr int kSettled = -1;
__device__ __forceinline__ int cap_range(const ScoreRules& r, float mx, bool counts = true)
{
    if (__all_sync(0xffffffffu, !counts || mx * r.near_in <= 1.f)) return 3;
    if (__all_sync(0xffffffffu, !counts || mx * r.mid_in <= 1.f)) return 2;
    return __all_sync(0xffffffffu, !counts || mx * r.wide_in <= 1.f) ? 1 : 0;
}

// Bits 0 .. n - 1 of a word (n is clamped to 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n)
{
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// The range of a tile that is cut and that with its hidden columns, outside [lo, hi), is none's.  What they hold does not
// count if a score lies beyond kNoScore caps, where tanh is 1 and none has a reason to be, or a lane has nothing but NaN:
// the range is then the one with zeros there.  (Short of that they may choose another form, within its error.  Without them in
// every case where the near range does not do: 64 sequences of 1024 tokens in documents of 200, 16 heads of 64, scores of
// deviation 3 under a cap of 30, 213 -> 270 us.)
constexpr float kNoScore = 10.f;
template <int N>
__device__ __forceinline__ int cap_range_seen(const ScoreRules& r, const float* s, float mx, int lo, int hi)
{
    if (__all_sync(0xffffffffu, mx * r.cap_in <= kNoScore)) return 0;
    float m = 0.f;
#pragma unroll
    for (int q = 0; q < N / 32; ++q) {
        const uint32_t see = low_bits(hi - 32 * q) & ~low_bits(lo - 32 * q);
#pragma unroll
        for (int c = 0; c < 32; ++c) m = fmaxf(m, (see >> c) & 1u ? fabsf(s[32 * q + c]) : 0.f);
    }
    return cap_range(r, m);
}

// Scores s of N keys under a cap, in base 2, in place.
template <int N>
__device__ __forceinline__ void capped_scores(float* s, const ScoreRules& r, int range, bool far)
{
    auto poly = [&](const auto& c) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 x = make_float2(s[i], s[i + 1]);
            const float2 y = __fmul2_rn(x, cap_factor(x, c));
            s[i] = y.x;
            s[i + 1] = y.y;
        }
    };
    if (range >= 2) poly(r.mid);
    else if (range == 1) poly(r.wide);
    else {
        if (range != kSettled) tanh_any<N>(s, r.cap_in, far);
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] *= r.mult;
    }
}

// s <- f(s) - slope * |dist - c| by pairs, for columns c = 0 .. N - 1 (dist: the position of the row less that of column
// 0).  sign = 1 where every column that counts lies at or before its row's position, -1 where behind it: the distance is
// then one sign's, counted on by eights.  0: either.  (Distances are whole numbers and exact.  Adding multiples of the
// slope instead is as fast, but the bias of a key next to the row is then off by the rounding of one a tile away.)
template <int N, typename F>
__device__ __forceinline__ void add_bias(float* s, float slope, float dist, int sign, F f)
{
    if (sign != 0) {
        const float2 sg = two(sign > 0 ? slope : -slope), eight = two(8.f);
        float2 d[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) d[h] = make_float2(static_cast<float>(2 * h) - dist, static_cast<float>(2 * h + 1) - dist);
#pragma unroll
        for (int c = 0; c < N; c += 8) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int i = c + 2 * h;
                const float2 y = __ffma2_rn(sg, d[h], f(make_float2(s[i], s[i + 1])));
                s[i] = y.x;
                s[i + 1] = y.y;
                if (c + 8 < N) d[h] = __fadd2_rn(d[h], eight);
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            const float2 y = f(make_float2(s[c], s[c + 1]));
            s[c] = fmaf(-slope, fabsf(dist - static_cast<float>(c)), y.x);
            s[c + 1] = fmaf(-slope, fabsf(dist - static_cast<float>(c + 1)), y.y);
        }
    }
}

// Scores s of N keys under a bias, and a cap if CAP, in place, over mult (as S and tanh are).
template <int N, bool CAP>
__device__ __forceinline__ void biased_scores(float* s, const ScoreRules& r, int range, bool far, float slope, float dist, int sign)
{
    if (CAP && range >= 2) {
        add_bias<N>(s, slope, dist, sign, [&](float2 x) { return __fmul2_rn(x, cap_factor(x, r.mid)); });
    } else {
        if (CAP && range != kSettled) tanh_any<N>(s, r.cap_in, far);
        add_bias<N>(s, slope, dist, sign, [&](float2 x) { return x; });
    }
}

// The largest of N numbers (a multiple of 32), NaN left out.
template <int N>
__device__ __forceinline__ float max_of(const float* s)
{
    float m[N / 32];
#pragma unroll
    for (int q = 0; q < N / 32; ++q) {
        const float* t = s + 32 * q;
        float a = max3(t[0], t[1], t[2]);
#pragma unroll
        for (int c = 3; c < 31; c += 2) a = max3(a, t[c], t[c + 1]);
        m[q] = fmaxf(a, t[31]);
    }
    if constexpr (N == 32) return m[0];
    else if constexpr (N == 64) return fmaxf(m[0], m[1]);
    else return max3(m[0], m[1], fmaxf(m[2], m[3]));
}

// Length of sequence b's prefix, 0 without any; out of range: clamped and recorded.
__device__ __forceinline__ int rules_prefix(const int* prefix, int b, int Nk, int* status)
{
    if (prefix == nullptr) return 0;
    const int x = prefix[b];
    if (x >= 0 && x <= Nk) return x;
    atomicCAS(status, 0, FA_ERR_INVALID_ARG);
    return min(max(x, 0), Nk);
}

}  // namespace fa
