// Eight neighbouring values of a row as FP32, from and to FP32, FP16 and 8-bit
// storage, for kernels that go over rows of any width and alignment.
//
// 8-bit values ("mx"): FP8 codes [rows, cols] and one scale for each 32 values of a
// row, [rows, ceil(cols / 32)] bytes; byte e stands for 2^(e - 127), 255 for NaN.
// The scale is the least power of two with max |x| / scale <= the format's largest
// value, the maximum over the finite values (1 where that is 0). So no finite value
// saturates, and a power of two costs an FP8 code no precision. Codes are rounded to
// nearest even. NaN gives a NaN code, and so do infinities in E4M3, which has none;
// in E5M2 they stay. FP16 values are first brought to the largest FP16 number with
// the format's mantissa (61440; 57344), so that what the codes stand for never
// rounds past FP16's range: off by less than half a step of the value.
#pragma once

#include "device_common.h"

namespace libgemm {

constexpr int kMxBlock = 32;

__device__ __forceinline__ float mx_scale(uint32_t e) {
    return bits_f32(e == 0u ? 0x00400000u : (e == 255u ? 0x7FC00000u : e << 23));
}

// Exponent (scale 2^e) for a block whose largest finite magnitude is m.
template <int FMT>
__device__ __forceinline__ int mx_exponent(float m) {
    // m = f 2^x, f in [0.5, 1); 448 = 0.875 2^9, 57344 = 0.875 2^16
    const int e = __builtin_amdgcn_frexp_expf(m) - (FMT == FMT_E5M2 ? 16 : 9) +
                  (__builtin_amdgcn_frexp_mantf(m) > 0.875f ? 1 : 0);
    return m > 0.0f ? max(e, -127) : 0;
}

// 2^e for e in [-127, 127].
__device__ __forceinline__ float mx_power(int e) { return mx_scale((uint32_t)(e + 127)); }

// Four codes of values / 2^e (given as mx_power) that are in the format's range,
// infinite or NaN. The scaled conversions round to nearest even (tested for every FP16
// value and every scale that holds it, and for FP32 values at every scale).
template <int FMT>
__device__ __forceinline__ uint32_t mx_pack4(float a, float b, float c, float d, float power) {
    typedef short v2s __attribute__((ext_vector_type(2)));
    v2s w = {0, 0};
    if constexpr (FMT == FMT_E5M2) {
        w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, a, b, power, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, c, d, power, true);
    } else {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, power, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, power, true);
    }
    return __builtin_bit_cast(uint32_t, w);
}

// The same of four FP16 values, two to a word.
template <int FMT>
__device__ __forceinline__ uint32_t mx_pack4_f16(uint32_t lo, uint32_t hi, float power) {
    typedef short v2s __attribute__((ext_vector_type(2)));
    typedef _Float16 v2hh __attribute__((ext_vector_type(2)));
    const v2hh a = __builtin_bit_cast(v2hh, lo), b = __builtin_bit_cast(v2hh, hi);
    v2s w = {0, 0};
    if constexpr (FMT == FMT_E5M2) {
        w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(w, a, power, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(w, b, power, true);
    } else {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, a, power, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, b, power, true);
    }
    return __builtin_bit_cast(uint32_t, w);
}

// Two codes of a word (its upper half: HI) times a scale.
template <int FMT, bool HI>
__device__ __forceinline__ auto mx_pair(uint32_t w, float scale) {
    if constexpr (FMT == FMT_E5M2) return __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, scale, HI);
    else return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, HI);
}

// |x| of a finite x, 0 of others.
__device__ __forceinline__ float finite_abs(float x) {
    const float a = __builtin_fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;
}

typedef v4u v4u_b1 __attribute__((aligned(1)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef v2u v2u_b1 __attribute__((aligned(1)));

// T: OUT_F32, OUT_F16, or OUT_E4M3 / OUT_E5M2 for codes (scaled by `scale`). n of
// the 8 values exist (others 0); vector accesses need no alignment.
template <int T>
__device__ __forceinline__ void load8(const void* base, int64_t at, int n, float scale, float (&v)[8]) {
    if (n >= 8) {
        if constexpr (T == OUT_F32) {
            const float* p = reinterpret_cast<const float*>(base) + at;
            const v4u a = *reinterpret_cast<const v4u_b1*>(p), b = *reinterpret_cast<const v4u_b1*>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = bits_f32(a[i]);
                v[4 + i] = bits_f32(b[i]);
            }
        } else if constexpr (T == OUT_F16) {
            const v8h a = __builtin_bit_cast(
                v8h, v4u(*reinterpret_cast<const v4u_b1*>(reinterpret_cast<const _Float16*>(base) + at)));
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
        } else {
            const v2u w = *reinterpret_cast<const v2u_b1*>(reinterpret_cast<const uint8_t*>(base) + at);
            constexpr int F = T == OUT_E5M2 ? FMT_E5M2 : FMT_E4M3;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const auto lo = mx_pair<F, false>(w[i], scale), hi = mx_pair<F, true>(w[i], scale);
                v[4 * i] = lo[0], v[4 * i + 1] = lo[1], v[4 * i + 2] = hi[0], v[4 * i + 3] = hi[1];
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = 0.0f;
        if (i >= n) continue;
        if constexpr (T == OUT_F32) v[i] = reinterpret_cast<const float*>(base)[at + i];
        else if constexpr (T == OUT_F16) v[i] = (float)reinterpret_cast<const _Float16*>(base)[at + i];
        else if constexpr (T == OUT_E5M2)
            v[i] = __builtin_amdgcn_cvt_pk_f32_bf8((int)reinterpret_cast<const uint8_t*>(base)[at + i], false)[0] * scale;
        else v[i] = __builtin_amdgcn_cvt_pk_f32_fp8((int)reinterpret_cast<const uint8_t*>(base)[at + i], false)[0] * scale;
    }
}

// A row in pieces of eight columns: piece c (c a multiple of 8) of a row of 8 columns
// and more is read and written whole. The last one, where the row cuts it, is the
// eight columns that end the row: the first `skip` of them are the piece's before it
// (whose lane computes and stores the same). skip of 8 and more: no piece.
struct Piece8 {
    int64_t at;
    int skip;
    __device__ __forceinline__ Piece8(int64_t c, int64_t width) : at(min(c, width - 8)), skip((int)min(c - at, (int64_t)8)) {}
};

// The values above in two steps, so that many loads can be in flight: eight whole
// values as they lie in memory, and what they are.
template <int T>
struct Raw8 {
    v4u w[T == OUT_F32 ? 2 : 1];   // (codes: two words)
    uint32_t e, before;            // the block's scale, and that of a cut piece's first `skip`
};

// CUT: rows that may cut a piece. Row r of `width` columns, scales of 8-bit values.
template <int T, bool CUT>
__device__ __forceinline__ void fetch8(Raw8<T>& x, const void* base, const uint8_t* scales, int64_t r, int64_t width,
                                       Piece8 p) {
    const int64_t at = r * width + p.at;
    if constexpr (T == OUT_F32) {
        const float* q = reinterpret_cast<const float*>(base) + at;
        x.w[0] = *reinterpret_cast<const v4u_b1*>(q);
        x.w[1] = *reinterpret_cast<const v4u_b1*>(q + 4);
    } else if constexpr (T == OUT_F16) {
        x.w[0] = *reinterpret_cast<const v4u_b1*>(reinterpret_cast<const _Float16*>(base) + at);
    } else {
        const v2u c = *reinterpret_cast<const v2u_b1*>(reinterpret_cast<const uint8_t*>(base) + at);
        x.w[0] = v4u{c[0], c[1], 0u, 0u};
        const uint8_t* s = scales + r * ((width + kMxBlock - 1) / kMxBlock);
        x.before = s[p.at / kMxBlock];
        x.e = CUT ? s[(p.at + 7) / kMxBlock] : x.before;
    }
}

template <int T, bool CUT>
__device__ __forceinline__ void values8(const Raw8<T>& x, int skip, float (&v)[8]) {
    if constexpr (T == OUT_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = bits_f32(x.w[i / 4][i % 4]);
    } else if constexpr (T == OUT_F16) {
        const v8h h = __builtin_bit_cast(v8h, x.w[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
    } else {
        constexpr int F = T == OUT_E5M2 ? FMT_E5M2 : FMT_E4M3;
        const float s = mx_scale(x.e), before = CUT ? mx_scale(x.before) : s;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const auto lo = mx_pair<F, false>(x.w[0][i], s), hi = mx_pair<F, true>(x.w[0][i], s);
            v[4 * i] = lo[0], v[4 * i + 1] = lo[1], v[4 * i + 2] = hi[0], v[4 * i + 3] = hi[1];
            if constexpr (CUT) {
                const auto lb = mx_pair<F, false>(x.w[0][i], before), hb = mx_pair<F, true>(x.w[0][i], before);
                v[4 * i] = 4 * i < skip ? lb[0] : lo[0], v[4 * i + 1] = 4 * i + 1 < skip ? lb[1] : lo[1];
                v[4 * i + 2] = 4 * i + 2 < skip ? hb[0] : hi[0], v[4 * i + 3] = 4 * i + 3 < skip ? hb[1] : hi[1];
            }
        }
    }
}

// Values of row r from column c (a multiple of 8) on; scales as above (8-bit only).
template <int T>
__device__ __forceinline__ void load_row8(const void* base, const uint8_t* scales, int64_t r, int64_t c, int64_t width,
                                          float (&v)[8]) {
    float s = 1.0f;
    if constexpr (T >= OUT_E4M3)
        s = c < width ? mx_scale(scales[r * ((width + kMxBlock - 1) / kMxBlock) + c / kMxBlock]) : 0.0f;
    const int64_t left = width - c;
    load8<T>(base, r * width + c, left >= 8 ? 8 : (left > 0 ? (int)left : 0), s, v);
}

// T: OUT_F32 or OUT_F16 (rounded to nearest even).
template <int T>
__device__ __forceinline__ void store8(void* base, int64_t at, int n, const float (&v)[8]) {
    if constexpr (T == OUT_F32) {
        float* p = reinterpret_cast<float*>(base) + at;
        if (n >= 8) {
            *reinterpret_cast<v4u_b1*>(p) = v4u{f32_bits(v[0]), f32_bits(v[1]), f32_bits(v[2]), f32_bits(v[3])};
            *reinterpret_cast<v4u_b1*>(p + 4) = v4u{f32_bits(v[4]), f32_bits(v[5]), f32_bits(v[6]), f32_bits(v[7])};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = v[i];
        }
    } else {
        _Float16* p = reinterpret_cast<_Float16*>(base) + at;
        v8h h;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
        if (n >= 8) {
            *reinterpret_cast<v4u_b1*>(p) = __builtin_bit_cast(v4u, h);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = h[i];
        }
    }
}

// Eight codes.
__device__ __forceinline__ void store_codes8(uint8_t* p, int n, uint32_t lo, uint32_t hi) {
    if (n >= 8) {
        *reinterpret_cast<v2u_b1*>(p) = v2u{lo, hi};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint8_t)((i < 4 ? lo >> (8 * i) : hi >> (8 * (i - 4))) & 0xFFu);
    }
}

// Sum and maximum over the 64 lanes of a wave (every lane has the result).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// (NaN in any lane: NaN.)
__device__ __forceinline__ float max_nan(float a, float b) { return a > b || a != a ? a : b; }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = max_nan(v, __shfl_xor(v, d, 64));
    return v;
}

}  // namespace libgemm
