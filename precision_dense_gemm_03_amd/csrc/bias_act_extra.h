// What the products with bias, activation and residual do with a tile's sums, in
// place of the plain kernels' scaling and store:
//
//   z = s acc + bias,  y = act(z) + residual,  C = y (FP8: y / sOut)
//
// s the scales' product, FP32 throughout; z itself is stored too where the backward
// pass wants it, as FP32 or FP16 or as 8-bit values (row_io.h), whose blocks of 32
// columns a wave holds whole. Types and activation are chosen at run time, once
// per tile and not per element: the kernels differ in their operands only.
#pragma once

#include "act.h"
#include "kernels.h"
#include "norm.h"
#include "row_io.h"

namespace libgemm {

// Which form of the activations (act.h) a kernel has: the one for FP16 and FP8
// results, the fine one for FP32 results, or both, chosen at run time. (Both in the
// ping-pong kernel cost its FP16 and FP8 results 1.4 to 2.7 %; in the others nothing,
// but 0.06 us of 11.3 for 4 rows of FP8.)
enum Fineness { COARSE = 0, FINE = 1, EITHER = 2 };

// apply(f), f(z) = activate(z) for the activation of a call.
template <int ACT, bool FINE>
struct Activate {
    __device__ __forceinline__ float operator()(float z) const { return activate<ACT, FINE>(z); }
};

template <int HOW, class F>
__device__ __forceinline__ void with_activation(int act, int out_dtype, F apply) {
    auto go = [&](auto fine) __attribute__((always_inline)) {
        constexpr bool fine_form = decltype(fine)::value;
        switch (act) {
            case ACT_GELU: apply(Activate<ACT_GELU, fine_form>{}); break;
            case ACT_GELU_TANH: apply(Activate<ACT_GELU_TANH, fine_form>{}); break;
            case ACT_SILU: apply(Activate<ACT_SILU, fine_form>{}); break;
            default: break;
        }
    };
    if (act == ACT_RELU) apply(Activate<ACT_RELU, false>{});
    else if (HOW == FINE || (HOW == EITHER && out_dtype == OUT_F32)) go(BoolC<true>{});
    else go(BoolC<false>{});
}

typedef unsigned int u32_b1 __attribute__((aligned(1)));

// LINES (ping-pong kernel): the FP16 residual and FP16 and FP32 results come and go
// past the caches, in whole 128-byte lines (16384 x 12288 x 4096 FP8 with bias and
// GELU_TANH 751 -> 707 us, with a residual too 808 -> 770: the caches' room is the
// operands').
template <bool LINES = false, int HOW = EITHER>
struct BiasActExtra {
    static constexpr bool kActive = false, kStores = false, kFinish = true;
    const float* sA;
    const float* sB;
    const float* sOut;       // FP8 outputs
    const float* bias;       // [N] or NULL
    const void* residual;    // [M, N] or NULL
    void* C;
    void* Z;                 // or NULL
    uint8_t* zscale;
    int act, res_dtype, out_dtype, z_dtype;
    int channel;             // sA[M] and sB[N], else one each (or NULL)

    // The factor of every element (per channel: beside sA[i] sB[j]).
    __device__ __forceinline__ float common() const { return channel ? 1.0f : (sA ? *sA : 1.0f) * (sB ? *sB : 1.0f); }
    // What y is multiplied by: y / sOut for FP8 outputs, in one factor (as the plain
    // products'), or in two where sOut is so small (2^-128) that its reciprocal is no FP32
    // number and a zero's product with it none. (rest is below 2^50 with the least sOut.)
    struct OutFactor {
        float lift, rest;
        __device__ __forceinline__ float operator()(float y) const { return y * lift * rest; }
    };
    __device__ __forceinline__ OutFactor out_factor() const {
        if (out_dtype < OUT_E4M3) return {1.0f, 1.0f};
        const float f = 1.0f / *sOut;
        if (__builtin_fabsf(f) < __builtin_inff()) return {1.0f, f};
        return {0x1p100f, 0x1p-100f / *sOut};
    }

    // Four neighbouring values of a row of FP32s, zero from N on.
    static __device__ __forceinline__ v4f row4(const float* p, int col, int N) {
        if (col + 4 <= N) return __builtin_bit_cast(v4f, v4u(*reinterpret_cast<const v4u_b1*>(p + col)));
        v4f v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = col + e < N ? p[col + e] : 0.0f;
        return v;
    }

    __device__ __forceinline__ v4f residual4(int row, int col, int N) const {
        const int64_t at = (int64_t)row * N;
        if (res_dtype == OUT_F32) return row4(reinterpret_cast<const float*>(residual) + at, col, N);
        const _Float16* p = reinterpret_cast<const _Float16*>(residual) + at + col;
        typedef _Float16 v4hh __attribute__((ext_vector_type(4)));
        v4f v;
        if (col + 4 <= N) {
            const v4hh h = __builtin_bit_cast(v4hh, v2u(*reinterpret_cast<const v2u_b1*>(p)));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (float)h[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = col + e < N ? (float)p[e] : 0.0f;
        }
        return v;
    }

    // Four neighbouring values to an [M, N] matrix of a type.
    static __device__ __forceinline__ void put4(void* base, int dtype, int row, int col, int N, v4f y) {
        const int64_t at = (int64_t)row * N + col;
        if (col + 4 <= N) {
            if (dtype == OUT_F32) {
                *reinterpret_cast<v4u_b1*>(reinterpret_cast<float*>(base) + at) = __builtin_bit_cast(v4u, y);
            } else if (dtype == OUT_F16) {
                typedef _Float16 v4hh __attribute__((ext_vector_type(4)));
                const v4hh h = {(_Float16)y[0], (_Float16)y[1], (_Float16)y[2], (_Float16)y[3]};
                *reinterpret_cast<v2u_b1*>(reinterpret_cast<_Float16*>(base) + at) = __builtin_bit_cast(v2u, h);
            } else {
                *reinterpret_cast<u32_b1*>(reinterpret_cast<uint8_t*>(base) + at) =
                    dtype == OUT_E5M2 ? e5m2_pack4(y[0], y[1], y[2], y[3]) : e4m3_pack4(y[0], y[1], y[2], y[3]);
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < N) store_out(base, at + e, y[e], dtype);
    }

    // 8-bit values of z: the block's exponent from its largest finite magnitude.
    __device__ __forceinline__ int exponent(float m) const {
        return z_dtype == OUT_E5M2 ? mx_exponent<FMT_E5M2>(m) : mx_exponent<FMT_E4M3>(m);
    }
    __device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float power) const {
        return z_dtype == OUT_E5M2 ? mx_pack4<FMT_E5M2>(a, b, c, d, power) : mx_pack4<FMT_E4M3>(a, b, c, d, power);
    }
    __device__ __forceinline__ void put_exponent(int row, int col, int N, int e) const {
        zscale[(int64_t)row * ((N + kMxBlock - 1) / kMxBlock) + col / kMxBlock] = (uint8_t)(e + 127);
    }

    // One element (decode kernel): z is scaled already.
    __device__ __forceinline__ void finish1(float z, int row, int col, int N) const {
        if (bias) z += bias[col];
        const int64_t at = (int64_t)row * N + col;
        if (Z) store_out(Z, at, z, z_dtype);
        float y = z;
        with_activation<HOW>(act, out_dtype, [&](auto f) __attribute__((always_inline)) { y = f(z); });
        if (residual)
            y += res_dtype == OUT_F32 ? reinterpret_cast<const float*>(residual)[at]
                                      : (float)reinterpret_cast<const _Float16*>(residual)[at];
        store_out(C, at, out_factor()(y), out_dtype);
    }

    // The deep-ring kernel: four neighbouring columns per lane and block, block tn at
    // columns col0 + 16 tn. Bias and residual are fetched before the K loop.
    struct Piece {
        v4f bias, residual;
    };

    __device__ __forceinline__ void prefetch(Piece& p, int row, int col, int kg, int M, int N) const {
        p.bias = p.residual = v4f{0.f, 0.f, 0.f, 0.f};
        if (kg != 0) return;
        if (bias) p.bias = row4(bias, col, N);
        if (residual && row < M) p.residual = residual4(row, col, N);
    }

    template <int TN>
    __device__ __forceinline__ void finish_ring(v4f (&acc)[TN], const Piece (&piece)[TN], int row, int col0, int M,
                                                int N) const {
        if (row >= M) return;
        const float s = common();
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) {
            acc[tn] *= s;
            if (channel) acc[tn] *= sA[row] * row4(sB, col0 + 16 * tn, N);
            acc[tn] += piece[tn].bias;
        }
        if (Z && z_dtype < OUT_E4M3) {
#pragma unroll
            for (int tn = 0; tn < TN; ++tn) put4(Z, z_dtype, row, col0 + 16 * tn, N, acc[tn]);
        } else if (Z) {
            // (the host asks only kernels for this whose waves hold 32 columns and more)
            if constexpr (TN >= 2) {
#pragma unroll
                for (int t = 0; t < TN; t += 2) {
                    float m = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float x = finite_abs(acc[t + e / 4][e % 4]);
                        if (col0 + 16 * (t + e / 4) + e % 4 < N) m = fmaxf(m, x);
                    }
                    m = fmaxf(m, __shfl_xor(m, 16, 64));
                    m = fmaxf(m, __shfl_xor(m, 32, 64));
                    const int e = exponent(m);
                    const float power = mx_power(e);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const v4f v = acc[t + u];
                        const uint32_t w = codes4(v[0], v[1], v[2], v[3], power);
                        const int col = col0 + 16 * (t + u);
                        uint8_t* p = reinterpret_cast<uint8_t*>(Z) + (int64_t)row * N + col;
                        if (col + 4 <= N) {
                            *reinterpret_cast<u32_b1*>(p) = w;
                        } else {
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                if (col + b < N) p[b] = (uint8_t)(w >> (8 * b));
                        }
                    }
                    // lanes 0 to 15 hold the block's first columns
                    if ((threadIdx.x & 63) < 16 && col0 + 16 * t < N) put_exponent(row, col0 + 16 * t, N, e);
                }
            }
        }
        with_activation<HOW>(act, out_dtype, [&](auto f) __attribute__((always_inline)) {
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[tn][e] = f(acc[tn][e]);
        });
        const OutFactor f = out_factor();
#pragma unroll
        for (int tn = 0; tn < TN; ++tn)
            put4(C, out_dtype, row, col0 + 16 * tn, N, (acc[tn] + piece[tn].residual) * f.lift * f.rest);
    }

    // The register-staged kernel: acc[tm][tn][r] is row row0 + 16 tm + r, column
    // col0 + 16 tn; the 16 lanes of a group hold neighbouring columns.
    template <int TM, int TN>
    __device__ __forceinline__ void finish_tile16(v4f (&acc)[TM][TN], int row0, int col0, int M, int N) const {
        static_assert(TN % 2 == 0, "blocks of 32 columns");
        const float s = common();
        const OutFactor f = out_factor();
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) {
            const int col = min(col0 + 16 * tn, N - 1);
            const float b = bias ? bias[col] : 0.0f, sb = channel ? sB[col] : 1.0f;
#pragma unroll
            for (int tm = 0; tm < TM; ++tm)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float v = acc[tm][tn][r] * s;
                    if (channel) v *= sA[min(row0 + 16 * tm + r, M - 1)] * sb;
                    acc[tm][tn][r] = v + b;
                }
        }
        if (Z && z_dtype < OUT_E4M3) {
#pragma unroll
            for (int tm = 0; tm < TM; ++tm)
#pragma unroll
                for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = row0 + 16 * tm + r, col = col0 + 16 * tn;
                        if (row < M && col < N) store_out(Z, (int64_t)row * N + col, acc[tm][tn][r], z_dtype);
                    }
        } else if (Z) {
#pragma unroll
            for (int tm = 0; tm < TM; ++tm)
#pragma unroll
                for (int t = 0; t < TN; t += 2)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = row0 + 16 * tm + r;
                        float m = 0.0f;
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            if (col0 + 16 * (t + u) < N) m = fmaxf(m, finite_abs(acc[tm][t + u][r]));
#pragma unroll
                        for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
                        const int e = exponent(m);
                        const float power = mx_power(e);
                        if (row >= M) continue;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int col = col0 + 16 * (t + u);
                            if (col < N)
                                reinterpret_cast<uint8_t*>(Z)[(int64_t)row * N + col] =
                                    (uint8_t)codes4(acc[tm][t + u][r], 0.0f, 0.0f, 0.0f, power);
                        }
                        if ((threadIdx.x & 15) == 0 && col0 + 16 * t < N) put_exponent(row, col0 + 16 * t, N, e);
                    }
        }
        with_activation<HOW>(act, out_dtype, [&](auto f) __attribute__((always_inline)) {
#pragma unroll
            for (int tm = 0; tm < TM; ++tm)
#pragma unroll
                for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[tm][tn][r] = f(acc[tm][tn][r]);
        });
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = row0 + 16 * tm + r, col = col0 + 16 * tn;
                    if (row >= M || col >= N) continue;
                    const int64_t at = (int64_t)row * N + col;
                    float y = acc[tm][tn][r];
                    if (residual)
                        y += res_dtype == OUT_F32 ? reinterpret_cast<const float*>(residual)[at]
                                                  : (float)reinterpret_cast<const _Float16*>(residual)[at];
                    store_out(C, at, f(y), out_dtype);
                }
    }

    // The ping-pong kernel (its acc, LDS regions and wave layout, gemm_pp_impl.h):
    // acc[i][j] holds row MR G + 32 i + lane % 32, columns 64 wj + 32 j + 8 q + 4
    // (lane / 32) + e in value 4 q + e. After the K loop the LDS is free: FP16 and
    // 8-bit values go through a wave's own part of it, so that memory is read and
    // written in 16-byte pieces of rows.
    //
    // A wave takes 32 of its rows through all steps and then the next 32, the sums
    // moving up, so that there is one copy of the code (one for each 32 rows, over 100
    // KB with every type's branches, waited for instructions; each step over all rows
    // at once spilled 593 registers). What M and N cut is read from clamped places and
    // not stored: a mask per store and none per read.
    template <int MI, class Lds>
    __device__ __forceinline__ void finish_pp(v16f (&acc)[MI][2], const Lds& lds, int m0, int n0, int G, int wj, int M,
                                              int cols) const {
        constexpr int MR = 32 * MI, STAGE = 64 * MI * 64;
        static_assert(STAGE >= 3 * kPart, "three parts of the wave's LDS");
        const int col0 = n0 + 64 * wj;   // of the wave's block
        if (col0 >= cols) return;
        LDS_AS uint8_t* ep = G == 0 ? (wj == 0 ? lds.b[0] : wj == 1 ? lds.b[1] : wj == 2 ? lds.b[2] : lds.b[3])
                                    : (wj < 2 ? lds.a[0] : lds.a[1]) + (wj & 1) * STAGE;
        const float s = common();
        const OutFactor f = out_factor();
        const bool res16 = residual && res_dtype == OUT_F16;
#pragma unroll 1
        for (int i = 0; i < MI; ++i) {
            const int row0 = m0 + MR * G + 32 * i;
            if (row0 >= M) break;
            // Nothing is carried from one 32 rows to the next but the sums: bias, scales,
            // addresses and masks of paths that a call does not take, kept over the loop,
            // spilled 250 registers. So they come from values made anew here.
            int lane = threadIdx.x & 63, N = cols;
            asm volatile("" : "+v"(lane), "+s"(N) : : "memory");
            const int lr = lane & 31, h = lane >> 5, lcol = col0 + 4 * h;   // this lane's columns: + 32 j + 8 q
            const int row = min(row0 + lr, M - 1);
            const bool whole = col0 + 64 <= N;
            v4u held[4];
            if (res16) fetch16(held, lane, row0, col0, M, N);
            float v[2][16];
            if (channel) {
                const float sa = sA[row];
                each_run(sB, lcol, N, whole, [&](int j, int q, v4f t) __attribute__((always_inline)) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[j][4 * q + e] = acc[0][j][4 * q + e] * (sa * t[e]);
                });
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[j][x] = acc[0][j][x] * s;
            }
            if (bias) {
                each_run(bias, lcol, N, whole, [&](int j, int q, v4f t) __attribute__((always_inline)) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[j][4 * q + e] += t[e];
                });
            }
            if (Z) {
                if (z_dtype >= OUT_E4M3) put_mx(v, ep, lane, row0, col0, M, N);
                else put_any(Z, z_dtype, v, ep, lane, row0, col0, M, N);
            }
            with_activation<HOW>(act, out_dtype, [&](auto f) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[j][x] = f(v[j][x]);
            });
            if (res16) {
                add16(v, held, ep + kPart, lane);
            } else if (residual) {
                each_run(reinterpret_cast<const float*>(residual) + (int64_t)row * N, lcol, N, whole,
                         [&](int j, int q, v4f t) __attribute__((always_inline)) {
#pragma unroll
                             for (int e = 0; e < 4; ++e) v[j][4 * q + e] += t[e];
                         });
            }
            if (out_dtype >= OUT_E4M3) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = f(v[j][4 * q + e]);
                        stage8(ep + 2 * kPart, lr, 32 * j + 8 * q + 4 * h,
                               out_dtype == OUT_E5M2 ? e5m2_pack4(y[0], y[1], y[2], y[3])
                                                     : e4m3_pack4(y[0], y[1], y[2], y[3]));
                    }
                drain8(reinterpret_cast<uint8_t*>(C), ep + 2 * kPart, lane, row0, col0, M, N);
            } else {
                put_any(C, out_dtype, v, ep + 2 * kPart, lane, row0, col0, M, N);
            }
#pragma unroll
            for (int k = 0; k + 1 < MI; ++k) {
                acc[k][0] = acc[k + 1][0];
                acc[k][1] = acc[k + 1][1];
            }
        }
    }

private:
    typedef _Float16 v4hh __attribute__((ext_vector_type(4)));
    static constexpr int kPart = 4096;   // 32 rows of 64 halves

    static __device__ __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

    // f(j, q, values) for the lane's eight runs of four columns of a row of FP32s;
    // what lies past N is some value of the row. whole: the wave's columns all exist.
    template <class F>
    static __device__ __forceinline__ void each_run(const float* p, int lcol, int N, bool whole, F f) {
        v4f t[8];
        if (whole || (N & 3) == 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                t[k] = __builtin_bit_cast(v4f, v4u(*reinterpret_cast<const v4u_b1*>(p + min(lcol + 32 * (k / 4) + 8 * (k % 4), N - 4))));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) t[k][e] = p[min(lcol + 32 * (k / 4) + 8 * (k % 4) + e, N - 1)];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) f(k / 4, k % 4, t[k]);
    }

    // 32 rows in LDS: 128 bytes a row, 16-byte chunk c of row r at slot c ^ (r / 2 % 8):
    // 32 rows at one column, or 8 rows whole, meet distinct banks.
    static __device__ __forceinline__ LDS_AS uint8_t* at16(LDS_AS uint8_t* ep, int r, int byte) {
        return ep + r * 128 + ((((byte >> 4) ^ ((r >> 1) & 7)) << 4) | (byte & 15));
    }

    // FP16 or FP32 values to an [M, N] matrix (FP32 32 columns at a time).
    static __device__ __forceinline__ void put_any(void* base, int dtype, const float (&v)[2][16], LDS_AS uint8_t* ep,
                                                   int lane, int row0, int col0, int M, int N) {
        const int lr = lane & 31, h = lane >> 5;
        if (dtype == OUT_F16) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v4hh x = {(_Float16)v[j][4 * q], (_Float16)v[j][4 * q + 1], (_Float16)v[j][4 * q + 2],
                                    (_Float16)v[j][4 * q + 3]};
                    *(LDS_AS v2i*)at16(ep, lr, 2 * (32 * j + 8 * q + 4 * h)) = __builtin_bit_cast(v2i, x);
                }
            drain16<2>(base, ep, lane, row0, col0, M, N);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *(LDS_AS v4f*)at16(ep, lr, 4 * (8 * q + 4 * h)) =
                        v4f{v[j][4 * q], v[j][4 * q + 1], v[j][4 * q + 2], v[j][4 * q + 3]};
                drain16<4>(base, ep, lane, row0, col0 + 32 * j, M, N);
            }
        }
    }

    // The LDS block's 32 rows of 128 bytes to memory, elements of ES bytes.
    template <int ES>
    static __device__ __forceinline__ void drain16(void* base, LDS_AS uint8_t* ep, int lane, int row0, int col0, int M, int N) {
        constexpr int VE = 16 / ES;
        const int seg = lane & 7, col = col0 + VE * seg;
        lds_done();
        uint8_t* d = reinterpret_cast<uint8_t*>(base) + ((int64_t)(row0 + (lane >> 3)) * N + col) * ES;
        v4u w[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) w[p] = *(const LDS_AS v4u*)at16(ep, 8 * p + (lane >> 3), 16 * seg);
#pragma unroll
        for (int p = 0; p < 4; ++p)
            if (row0 + 8 * p + (lane >> 3) < M && col + VE <= N) {
                if constexpr (LINES) __builtin_nontemporal_store(w[p], reinterpret_cast<v4u*>(d + (int64_t)(8 * p) * N * ES));
                else *reinterpret_cast<v4u_b1*>(d + (int64_t)(8 * p) * N * ES) = w[p];
            }
        if (N % VE != 0) {   // the piece that ends a row
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (row0 + 8 * p + (lane >> 3) < M && col + e < N && col + VE > N) {
                        uint8_t* at = d + ((int64_t)(8 * p) * N + e) * ES;
                        if constexpr (ES == 4) *reinterpret_cast<uint32_t*>(at) = w[p][e];
                        else *reinterpret_cast<uint16_t*>(at) = (uint16_t)(w[p][e / 2] >> (16 * (e & 1)));
                    }
        }
        lds_done();   // the block may be written again
    }

    // 32 rows of the FP16 residual, in 16-byte pieces of rows.
    __device__ __forceinline__ void fetch16(v4u (&held)[4], int lane, int row0, int col0, int M, int N) const {
        const int col = col0 + 8 * (lane & 7);
        const bool whole = col0 + 64 <= N;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const _Float16* s =
                reinterpret_cast<const _Float16*>(residual) + (int64_t)min(row0 + 8 * p + (lane >> 3), M - 1) * N;
            if (whole || (N & 7) == 0) {
                if constexpr (LINES) held[p] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(s + min(col, N - 8)));
                else held[p] = *reinterpret_cast<const v4u_b1*>(s + min(col, N - 8));
            } else {
                v8h x;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = s[min(col + e, N - 1)];
                held[p] = __builtin_bit_cast(v4u, x);
            }
        }
    }

    static __device__ __forceinline__ void add16(float (&v)[2][16], const v4u (&held)[4], LDS_AS uint8_t* ep, int lane) {
        const int lr = lane & 31, h = lane >> 5;
#pragma unroll
        for (int p = 0; p < 4; ++p) *(LDS_AS v4u*)at16(ep, 8 * p + (lane >> 3), 16 * (lane & 7)) = held[p];
        lds_done();
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const v4hh r = __builtin_bit_cast(v4hh, *(const LDS_AS v2i*)at16(ep, lr, 2 * (32 * j + 8 * q + 4 * h)));
#pragma unroll
                for (int e = 0; e < 4; ++e) v[j][4 * q + e] += (float)r[e];
            }
        lds_done();
    }

    // 32 rows of codes in LDS: 64 bytes a row, chunk c of row r at slot c ^ (r / 4 % 4).
    static __device__ __forceinline__ void stage8(LDS_AS uint8_t* ep, int r, int byte, uint32_t w) {
        *(LDS_AS uint32_t*)(ep + r * 64 + ((((byte >> 4) ^ ((r >> 2) & 3)) << 4) | (byte & 15))) = w;
    }

    static __device__ __forceinline__ void drain8(uint8_t* base, LDS_AS uint8_t* ep, int lane, int row0, int col0, int M, int N) {
        const int seg = lane & 3, col = col0 + 16 * seg;
        lds_done();
        uint8_t* d = base + (int64_t)(row0 + (lane >> 2)) * N + col;
        v4u w[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int r = 16 * p + (lane >> 2);
            w[p] = *(const LDS_AS v4u*)(ep + r * 64 + 16 * (seg ^ ((r >> 2) & 3)));
        }
#pragma unroll
        for (int p = 0; p < 2; ++p)
            if (row0 + 16 * p + (lane >> 2) < M && col + 16 <= N) *reinterpret_cast<v4u_b1*>(d + (int64_t)(16 * p) * N) = w[p];
        if ((N & 15) != 0) {
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (row0 + 16 * p + (lane >> 2) < M && col + e < N && col + 16 > N)
                        d[(int64_t)(16 * p) * N + e] = (uint8_t)(w[p][e / 4] >> (8 * (e % 4)));
        }
        lds_done();
    }

    // 8-bit values of z: a row's block of 32 columns is in two lanes.
    __device__ __forceinline__ void put_mx(float (&v)[2][16], LDS_AS uint8_t* ep, int lane, int row0, int col0, int M,
                                           int N) const {
        const int lr = lane & 31, h = lane >> 5, row = row0 + lr;
        if (col0 + 64 > N) {   // columns past N take no part
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    v[j][x] = col0 + 32 * j + 8 * (x >> 2) + 4 * h + (x & 3) < N ? v[j][x] : 0.0f;
        }
        uint32_t both = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float m = 0.0f;
#pragma unroll
            for (int x = 0; x < 16; ++x) m = fmaxf(m, __builtin_fabsf(v[j][x]));
            if (__builtin_amdgcn_ballot_w64(!(m < __builtin_inff())) != 0) {   // (fmaxf passes NaN over)
                m = 0.0f;
#pragma unroll
                for (int x = 0; x < 16; ++x) m = fmaxf(m, finite_abs(v[j][x]));
            }
            m = fmaxf(m, __shfl_xor(m, 32, 64));
            const int e = exponent(m);
            const float power = mx_power(e);
            both |= (uint32_t)(e + 127) << (8 * j);
            if (z_dtype == OUT_E5M2) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    stage8(ep, lr, 32 * j + 8 * q + 4 * h,
                           mx_pack4<FMT_E5M2>(v[j][4 * q], v[j][4 * q + 1], v[j][4 * q + 2], v[j][4 * q + 3], power));
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    stage8(ep, lr, 32 * j + 8 * q + 4 * h,
                           mx_pack4<FMT_E4M3>(v[j][4 * q], v[j][4 * q + 1], v[j][4 * q + 2], v[j][4 * q + 3], power));
            }
        }
        // lane h of a row stores the scale of its half of the columns
        const int col = col0 + 32 * h;
        if (row < M && col < N)
            zscale[(int64_t)row * ((N + kMxBlock - 1) / kMxBlock) + col / kMxBlock] = (uint8_t)(both >> (8 * h));
        drain8(reinterpret_cast<uint8_t*>(Z), ep, lane, row0, col0, M, N);
    }
};

template <bool LINES = false, int HOW = EITHER>
BiasActExtra<LINES, HOW> bias_act_extra(const BiasActArgs& a) {
    return BiasActExtra<LINES, HOW>{a.sA, a.sB, a.sOut, a.bias, a.residual, a.C, a.Z, a.zscale, a.act, a.res_dtype,
                                    a.out_dtype, a.z_dtype, a.channel};
}

}  // namespace libgemm
