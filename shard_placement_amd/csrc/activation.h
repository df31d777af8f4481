// activation.h -- activation functions and their slopes in binary32, shared by
// the layer products (linear.hip) and the gated block (gated.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "tide.h"

namespace tide {

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kLog2E = 1.4426950408889634f;
// 2 sqrt(2 / pi) (z + 0.044715 z^3) = z (kTanhC + kTanhA z^2)
constexpr float kTanhC = 1.5957691216057308f;
constexpr float kTanhA = kTanhC * 0.044715f;

// 1 / (1 + exp(-u)), off by a few binary32 steps; 0.5 (1 + tanh(v)) is this at
// u = 2 v, so the tanh form of gelu is z * sigmoid(z (kTanhC + kTanhA z^2)).
// The exponential's and the reciprocal's instructions are within one step; a
// division written out would be most of the epilogue's work.
__device__ __forceinline__ float sigmoid(float u) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * u));
}

// exp(-z^2 / 2) and the normal distribution's Phi(z).  Its lower tail is
// erfc(x) / 2, x = |z| / sqrt(2), and erfc(x) = t Q(t) exp(-x^2) with t = 1 / (1 +
// 0.375 x).  Q is fitted to the least relative error over 0 <= x <= 10 (6.4e-7;
// from x = 9.3 on exp(-x^2) is below binary32's normal numbers and 0 here), so
// gelu is a bf16 rounding off in its far negative tail too, where a formula of
// small absolute error is percents off.  A library erff took 55 us in the
// gradient of 2048 x 13824 elements, which reads and writes 141 MB, where this
// takes 39; a forward of 4096 x 16384 x 1024 with gelu takes 157 us, 154 with
// a shorter polynomial of small absolute error, 2% off at z = -10.
__device__ __forceinline__ float normal_cdf(float z, float* bell) {
    const float g = __builtin_amdgcn_exp2f(-0.5f * kLog2E * (z * z));
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.375f * kSqrtHalf, fabsf(z), 1.0f));
    float poly = __builtin_fmaf(-0.1350946333f, t, 0.3879334708f);
    poly = __builtin_fmaf(poly, t, -0.1295913167f);
    poly = __builtin_fmaf(poly, t, 0.2830573515f);
    poly = __builtin_fmaf(poly, t, 0.1666661391f);
    poly = __builtin_fmaf(poly, t, 0.2156888808f);
    poly = __builtin_fmaf(poly, t, 0.2113394712f);
    const float tail = 0.5f * poly * t * g;
    *bell = g;
    return z < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == TIDE_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    if constexpr (ACT == TIDE_ACT_GELU) {
        float bell;
        return z * normal_cdf(z, &bell);
    }
    if constexpr (ACT == TIDE_ACT_GELU_TANH)
        return z * sigmoid(z * __builtin_fmaf(kTanhA, z * z, kTanhC));
    if constexpr (ACT == TIDE_ACT_SILU) return z * sigmoid(z);
    return z;
}

// z may be infinite where a finite one was kept (act8.h: values that round up
// to 2^128), and infinity times the 0 that bounds it would be NaN: a factor z is
// held within what changes nothing, the other factor being 0 outside.  (NaN
// reaches the result through the other terms.)
__device__ __forceinline__ float within(float z) { return __builtin_amdgcn_fmed3f(z, -256.0f, 256.0f); }

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == TIDE_ACT_RELU) return z > 0.0f ? 1.0f : z < 0.0f ? 0.0f : 0.0f * z;
    if constexpr (ACT == TIDE_ACT_GELU) {
        float bell;
        const float cdf = normal_cdf(z, &bell);
        return __builtin_fmaf(within(z) * kInvSqrt2Pi, bell, cdf);
    }
    if constexpr (ACT == TIDE_ACT_GELU_TANH) {
        const float t = z * z;
        const float s = sigmoid(z * __builtin_fmaf(kTanhA, t, kTanhC));
        // where the sigmoid is 0 or 1 the polynomial may be infinite already
        const float q = __builtin_fmaf(-s, s, s);
        return q > 0.0f ? __builtin_fmaf(z * q, __builtin_fmaf(3.0f * kTanhA, t, kTanhC), s) : s;
    }
    if constexpr (ACT == TIDE_ACT_SILU) {
        const float s = sigmoid(z);
        return s * __builtin_fmaf(within(z), 1.0f - s, 1.0f);
    }
    return 1.0f;
}

// act(z) and act'(z) together, for a z that was kept: where it reads back as minus
// infinity act's limit is 0, not infinity times 0.
template <int ACT>
__device__ __forceinline__ float act_both(float z, float* slope) {
    if constexpr (ACT == TIDE_ACT_GELU || ACT == TIDE_ACT_GELU_TANH || ACT == TIDE_ACT_SILU) {
        const float low = z < -256.0f ? -256.0f : z;  // NaN stays NaN
        if constexpr (ACT == TIDE_ACT_GELU) {
            float bell;
            const float cdf = normal_cdf(z, &bell);
            *slope = __builtin_fmaf(within(z) * kInvSqrt2Pi, bell, cdf);
            return low * cdf;
        } else if constexpr (ACT == TIDE_ACT_GELU_TANH) {
            const float t = z * z;
            const float s = sigmoid(z * __builtin_fmaf(kTanhA, t, kTanhC));
            const float q = __builtin_fmaf(-s, s, s);
            *slope = q > 0.0f ? __builtin_fmaf(z * q, __builtin_fmaf(3.0f * kTanhA, t, kTanhC), s) : s;
            return low * s;
        } else {
            const float s = sigmoid(z);
            *slope = s * __builtin_fmaf(within(z), 1.0f - s, 1.0f);
            return low * s;
        }
    }
    *slope = act_slope<ACT>(z);
    return act_value<ACT>(z);
}

// v to act(v), eight at a time: the choice is made once for all of them.
template <int ACT>
__device__ __forceinline__ void apply_act(float (&v)[8]) {
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = act_value<ACT>(v[r]);
}
__device__ __forceinline__ void apply_act(float (&v)[8], int act) {
    switch (act) {
        case TIDE_ACT_RELU: return apply_act<TIDE_ACT_RELU>(v);
        case TIDE_ACT_GELU: return apply_act<TIDE_ACT_GELU>(v);
        case TIDE_ACT_GELU_TANH: return apply_act<TIDE_ACT_GELU_TANH>(v);
        case TIDE_ACT_SILU: return apply_act<TIDE_ACT_SILU>(v);
        default: return;
    }
}

// v times act'(z).
template <int ACT>
__device__ __forceinline__ void apply_slope(const float (&z)[8], float (&v)[8]) {
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] *= act_slope<ACT>(z[r]);
}

}  // namespace tide
