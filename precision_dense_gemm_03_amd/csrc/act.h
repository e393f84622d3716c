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
// P(-a), a >= 0, is 2 to the power of a polynomial in a (activate), fitted here for
// the least error over [0, 7]: 7e-7 of P, and with FP32's rounding of the exponent,
// which grows to 40, 4.5e-6; beyond 7, where P is below 1.3e-12, it falls to 0. The
// derivative needs exp(-a^2 / 2) as well, so there P(-a) is exp(-a^2 / 2) times a
// function that falls from 1/2 like 1 / (a sqrt(2 pi)): a polynomial without constant
// in t = 1 / (1 + 0.35 a), fitted here for the least relative error over a in [0, 7]:
// 2.5e-7 there, 4.5e-5 beyond, where P is below 1.3e-12. So small tails keep their
// relative precision; the exponent's rounding adds a^2 2^-24.
#pragma once

#include "device_common.h"

namespace libgemm {

enum Activation { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhScale = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

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

// 1 / (1 + 2^u)
__device__ __forceinline__ float logistic2(float u) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u)); }

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == ACT_RELU) {
        return z < 0.0f ? 0.0f : z;
    } else if constexpr (ACT == ACT_GELU) {
        const float q = normal_below(__builtin_fabsf(z));
        return z * (z < 0.0f ? q : 1.0f - q);
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
