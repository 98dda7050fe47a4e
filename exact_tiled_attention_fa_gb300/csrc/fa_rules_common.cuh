// fa_rules_common.cuh -- what the kernels of attention under score rules share.
//
// Scores.  With x = scale q.k, a cap c > 0 makes it c tanh(x / c), whose slope is 1 - tanh^2; a bias then takes
// slope_h |i - j| off (i, j the positions of query and key).  In base 2, as the exponentials want them:
// mult * tanh(cap_in * S) - slope2 * |i - j|, S = q.k.
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

// tanh of N numbers k * s, in place.  Arguments up to kTanhRange, where scores that a cap is meant for almost
// always are, take an odd polynomial on the FMA units: u P(u^2) with P the minimax polynomial of degree 5 for
// tanh(u) / u (Remez exchange on u^2 in [0, 0.5625], relative error 2.9e-8).  Others take 1 - 2 / (1 + e^2u), two
// operations of the special function unit that the softmax's exponentials also need; its absolute error of 2e-7
// is one of 1e-5 of a weight at a cap of 50.  +-infinity gives +-1, NaN NaN.  (The device's own tanh instruction
// is off by 2^-11 of its result: at a score of 20 by 0.01, and the weight by as much.) 
constexpr float kTanhRange = 0.75f;

template <int N>
__device__ __forceinline__ void tanh_small(float* s, float k)
{
    constexpr float c0 = 0.99999997101f, c1 = -0.3333295888f, c2 = 0.13325406021f, c3 = -0.053344430265f, c4 = 0.019582908378f,
                    c5 = -0.0047162573577f;
    auto two = [](float x) { return make_float2(x, x); };
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const float2 u = __fmul2_rn(make_float2(s[c], s[c + 1]), two(k));
        const float2 w = __fmul2_rn(u, u);
        float2 q = __ffma2_rn(w, two(c5), two(c4));
        q = __ffma2_rn(w, q, two(c3));
        q = __ffma2_rn(w, q, two(c2));
        q = __ffma2_rn(w, q, two(c1));
        q = __ffma2_rn(w, q, two(c0));
        q = __fmul2_rn(u, q);
        s[c] = q.x;
        s[c + 1] = q.y;
    }
}

template <int N>
__device__ __forceinline__ void tanh_any(float* s, float k)
{
    const float k2 = k * (2.f * kLog2e);
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] = fmaf(-2.f, rcp_approx(1.f + ex2(s[c] * k2)), 1.f);
}

// s <- mult * s - slope2 * |dist - c| for columns c = 0 .. N - 1 (dist: the position of the row less that of column
// 0).  sign = 1 where every column lies at or before its row's position, -1 where behind it: the bias is then linear
// in c, a start for each 32 columns and steps of 8 added to it (four roundings).  0: either.
template <int N>
__device__ __forceinline__ void add_bias(float* s, float mult, float slope2, float dist, int sign)
{
    const float2 m2 = make_float2(mult, mult);
    if (sign != 0) {
        const float sg = sign > 0 ? slope2 : -slope2;
        const float base = -sg * dist;
        const float2 step = make_float2(8.f * sg, 8.f * sg);
#pragma unroll
        for (int c0 = 0; c0 < N; c0 += 32) {
            float2 b[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) b[h] = make_float2(fmaf(static_cast<float>(c0 + 2 * h), sg, base), fmaf(static_cast<float>(c0 + 2 * h + 1), sg, base));
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int i = c0 + c + 2 * h;
                    const float2 y = __ffma2_rn(make_float2(s[i], s[i + 1]), m2, b[h]);
                    s[i] = y.x;
                    s[i + 1] = y.y;
                    if (c + 8 < 32) b[h] = __fadd2_rn(b[h], step);
                }
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] = fmaf(-slope2, fabsf(dist - static_cast<float>(c)), s[c] * mult);
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

// Bits 0 .. n - 1 of a word (n is clamped to 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n)
{
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
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
