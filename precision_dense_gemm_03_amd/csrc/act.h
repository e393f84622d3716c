// Activations of a product's epilogue and their derivatives, in FP32.
//
//   RELU       max(z, 0)
//   GELU       z P(z), P the normal distribution function
//   GELU_TANH  z s(2 sqrt(2/pi) (z + 0.044715 z^3)), s(u) = 1 / (1 + exp(-u)):
//              0.5 z (1 + tanh(u / 2)) with one exponential
//   SILU       z s(z)
// NaN gives NaN (RELU's derivative: 0); +inf gives +inf, and -inf NaN where the
// formula is -inf * 0. Derivatives at infinities are their limits, 1 and 0.
//
// Two forms of each function (FINE). An FP32 result keeps FP32's precision over the
// whole range, small tails among it: arguments of exponentials are held in two FP32
// numbers, and GELU's P(-a), a >= 0, is exp(-a^2 / 2) times a function that falls from
// 1/2 like 1 / (a sqrt(2 pi)), fitted here as a polynomial without constant in t = 1 /
// (1 + 0.35 a): 6.7e-8 over [0, 13.5] with its coefficients in FP32. In all GELU is
// within 4.2e-7 of its value, SILU and GELU_TANH within 2.2e-7.
//
// Results that are rounded to FP16 or FP8 (half a step of 4.9e-4 and more) take shorter
// forms (4096^3 FP16 into FP32, us: GELU 127 with them and 131 with the fine ones,
// GELU_TANH 124 and 132, SILU 124 and 126): arguments of exponentials are rounded to
// FP32, which costs a value their size times 2^-24, and P(-a) is 2 to the power of a
// polynomial in a, fitted here over [0, 7]: with its coefficients in FP32 off by 1.4e-6
// of P, evaluated in FP32 by 5.2e-6 (1.4e-6 below 3); beyond 7, where P is below
// 1.3e-12, it falls to 0.
//
// The derivative needs exp(-a^2 / 2) as well; there P(-a) is of the fine form with a
// shorter polynomial: 2.7e-7 over [0, 7], 4.5e-5 beyond. Small tails keep their
// relative precision; the exponent's roundings add up to 1.5 a^2 2^-24.
#pragma once

#include "device_common.h"

namespace libgemm {

enum Activation { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhScale = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// A constant as the sum of two FP32 numbers.
struct TwoFloats {
    float hi, lo;
};
constexpr TwoFloats two_floats(double c) { return {(float)c, (float)(c - (double)(float)c)}; }

// exp(-a^2 / 2) and P(-a) for a = |z|.
__device__ __forceinline__ float normal_tail(float a, float& e) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.35f, 1.0f));
    e = __builtin_amdgcn_exp2f((a * a) * (-0.5f * kLog2e));
    float p = 0.0474968888f;
    p = __builtin_fmaf(p, t, -0.195784926f);
    p = __builtin_fmaf(p, t, 0.229083672f);
    p = __builtin_fmaf(p, t, -0.00567076728f);
    p = __builtin_fmaf(p, t, 0.149493217f);
    p = __builtin_fmaf(p, t, 0.13548772f);
    p = __builtin_fmaf(p, t, 0.139894322f);
    return p * t * e;
}

__device__ __forceinline__ float normal_below(float a) {
    float p = -5.7345082e-09f;
    p = __builtin_fmaf(p, a, 2.15684988e-07f);
    p = __builtin_fmaf(p, a, -3.38793217e-06f);
    p = __builtin_fmaf(p, a, 2.72261461e-05f);
    p = __builtin_fmaf(p, a, -8.73539296e-05f);
    p = __builtin_fmaf(p, a, -0.000462577848f);
    p = __builtin_fmaf(p, a, 0.00762082624f);
    p = __builtin_fmaf(p, a, -0.0530025812f);
    p = __builtin_fmaf(p, a, -0.458984411f);
    p = __builtin_fmaf(p, a, -1.15114265f);
    p = __builtin_fmaf(p, a, -0.999998975f);
    return __builtin_amdgcn_exp2f(p);
}

// 2^(x + low) for a low that is small beside 1. (An infinity stays one.)
__device__ __forceinline__ float exp2_fine(float x, float low) {
    return __builtin_amdgcn_exp2f(x) * __builtin_fmaf(low, 0.6931471805599453f, 1.0f);
}

// P(-a) with FP32's precision. (Where a passes 100 it is 0.)
__device__ __forceinline__ float normal_below_fine(float a) {
    a = fminf(a, 100.0f);
    constexpr TwoFloats c = two_floats(-0.5 * 1.4426950408889634);
    const float s = a * a, x = s * c.hi;
    float low = __builtin_fmaf(s, c.hi, -x);
    low = __builtin_fmaf(s, c.lo, low);
    low = __builtin_fmaf(__builtin_fmaf(a, a, -s), c.hi, low);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.35f, 1.0f));
    float p = -0.029125856f;
    p = __builtin_fmaf(p, t, 0.1438722f);
    p = __builtin_fmaf(p, t, -0.2555045f);
    p = __builtin_fmaf(p, t, 0.15892924f);
    p = __builtin_fmaf(p, t, -0.022937113f);
    p = __builtin_fmaf(p, t, 0.10543293f);
    p = __builtin_fmaf(p, t, 0.11985244f);
    p = __builtin_fmaf(p, t, 0.13985908f);
    p = __builtin_fmaf(p, t, 0.13962157f);
    return p * t * exp2_fine(x, low);
}

// -log2(e) times SILU's argument and the tanh form's, as x + low. v is of at most 100
// in magnitude, so that nothing passes FP32's range.
__device__ __forceinline__ void silu_exponent(float v, float& x, float& low) {
    constexpr TwoFloats c = two_floats(-1.4426950408889634);
    x = v * c.hi;
    low = __builtin_fmaf(v, c.lo, __builtin_fmaf(v, c.hi, -x));
}

__device__ __forceinline__ void tanh_exponent(float v, float& x, float& low) {
#pragma clang fp contract(off)   // (p is the rounded product wherever it stands)
    constexpr double scale = -1.4426950408889634 * 1.5957691216057308;
    constexpr TwoFloats c1 = two_floats(scale), c3 = two_floats(scale * 0.044715);
    const float w = v * v, p = w * c3.hi;
    float pl = __builtin_fmaf(w, c3.hi, -p);
    pl = __builtin_fmaf(w, c3.lo, pl);
    pl = __builtin_fmaf(__builtin_fmaf(v, v, -w), c3.hi, pl);
    const float k = c1.hi + p, b = k - c1.hi;   // k and what its rounding left
    const float kl = (c1.hi - (k - b)) + (p - b) + (pl + c1.lo);
    x = v * k;
    low = __builtin_fmaf(v, kl, __builtin_fmaf(v, k, -x));
}

// 1 / (1 + 2^u)
__device__ __forceinline__ float logistic2(float u) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u)); }

template <int ACT, bool FINE>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == ACT_RELU) {
        return z < 0.0f ? 0.0f : z;
    } else if constexpr (ACT == ACT_GELU) {
        const float a = __builtin_fabsf(z), q = FINE ? normal_below_fine(a) : normal_below(a);
        return z * (z < 0.0f ? q : 1.0f - q);
    } else if constexpr (FINE && (ACT == ACT_GELU_TANH || ACT == ACT_SILU)) {
        const float v = fminf(fmaxf(z, -100.0f), 100.0f);   // (NaN: z itself keeps it)
        float x, low;
        if constexpr (ACT == ACT_SILU) silu_exponent(v, x, low);
        else tanh_exponent(v, x, low);
        return z * __builtin_amdgcn_rcpf(1.0f + exp2_fine(x, low));
    } else if constexpr (ACT == ACT_GELU_TANH) {
        return z * logistic2(z * __builtin_fmaf(z * z, -kLog2e * kTanhScale * kTanhCubic, -kLog2e * kTanhScale));
    } else if constexpr (ACT == ACT_SILU) {
        return z * logistic2(z * -kLog2e);
    } else {
        return z;
    }
}

// The derivative. (1 - s is exp(-u) s: the difference would lose its bits.
// Exponents stop at 2^115, where s is 0 against every other term, z standing for no
// more than 1000 in magnitude: beyond, the derivative is 0 or 1 and z^3 may not be a
// number. Selects, which keep NaN.)
template <int ACT>
__device__ __forceinline__ float slope(float z) {
    if constexpr (ACT == ACT_GELU || ACT == ACT_GELU_TANH || ACT == ACT_SILU) {
        z = z > 1000.0f ? 1000.0f : z;
        z = z < -1000.0f ? -1000.0f : z;
    }
    if constexpr (ACT == ACT_RELU) {
        return z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == ACT_GELU) {
        float e;
        const float q = normal_tail(__builtin_fabsf(z), e);
        return __builtin_fmaf(z * 0.3989422804014327f, e, z < 0.0f ? q : 1.0f - q);
    } else if constexpr (ACT == ACT_GELU_TANH || ACT == ACT_SILU) {
        const float zz = z * z;
        const float u = ACT == ACT_SILU ? z : z * __builtin_fmaf(zz, kTanhScale * kTanhCubic, kTanhScale);
        const float e = __builtin_amdgcn_exp2f(fminf(u * -kLog2e, 115.0f));
        const float s = __builtin_amdgcn_rcpf(1.0f + e);
        const float du = ACT == ACT_SILU ? 1.0f : __builtin_fmaf(zz, 3.0f * kTanhScale * kTanhCubic, kTanhScale);
        return s * __builtin_fmaf(z * du, e * s, 1.0f);
    } else {
        return 1.0f;
    }
}

}  // namespace libgemm
