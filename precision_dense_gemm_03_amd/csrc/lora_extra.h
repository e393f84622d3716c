// The low-rank term of a product with per-row adapters, added to a tile's
// accumulators after its K loop (lora.hip computes the low-rank values):
//
//   y[i, j] = base[i, j] + sum_r low[i, r] LB[a_i, j, r],   a_i the row's adapter
//
// low is FP32 and LB FP16, so each row's low values are split into two FP16
// numbers, hi + lo, of 22 bits together, after scaling the row's piece of 64
// by a power of two that puts its largest value into [2^14, 2^15): the split
// then drops at most 2^-22 of that largest value (lo rounds to half a step,
// 2^-11 of hi's half step), below FP32's own rounding of the sums it came from
// for any K above 16. The scaling is undone on the FP32 sum, exactly. Both
// halves meet LB's operand, loaded once, on the matrix cores.
//
// Rows of one block may have several adapters: each adapter present multiplies
// the whole block and only its rows take the sum, so no other adapter's values
// (NaN included) reach a row.
#pragma once

#include "device_common.h"

namespace libgemm {

struct LoraExtra {
    static constexpr bool kActive = true;
    const float* low;         // [rows, rank_p], zero from rank on
    const int32_t* adapter;   // [rows]
    const _Float16* LB;       // [adapters, N, rank]
    int rank, rank_p;         // rank_p: rank rounded up to a multiple of 8
    int adapters;

    __device__ __forceinline__ int adapter_of(int row, int M) const {
        const int a = row < M ? adapter[row] : -1;
        return a >= 0 && a < adapters ? a : -1;
    }

    // Eight values of one row of LB from r0 on, zero from rank on.
    __device__ __forceinline__ v8h lb_chunk(int a, int col, int r0, int N) const {
        typedef v4u any16 __attribute__((aligned(2)));
        const _Float16* p = LB + ((int64_t)a * N + col) * rank;
        if (r0 + 8 <= rank) return __builtin_bit_cast(v8h, *reinterpret_cast<const any16*>(p + r0));
        v8h v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = r0 + i < rank ? p[r0 + i] : (_Float16)0.0f;
        return v;
    }

    // This lane's STEPS chunks of a row's piece [p0, p0 + 64) as hi and lo
    // operands; chunk s is 8 (GROUPS s + g) values into the piece, and the
    // lanes that share the row differ in lane bits 64 / GROUPS and up. Returns
    // the piece's exponent.
    template <int STEPS, int GROUPS>
    __device__ __forceinline__ int split_piece(const float* row, int p0, int g, v8h (&hi)[STEPS],
                                               v8h (&lo)[STEPS]) const {
        float v[STEPS][8];
        float m = 0.0f;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int r0 = p0 + 8 * (GROUPS * s + g);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4f t = v4f{0.f, 0.f, 0.f, 0.f};
                if (r0 < rank_p) t = *reinterpret_cast<const v4f*>(row + r0 + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[s][4 * h + i] = t[i];
                    m = fmaxf(m, __builtin_fabsf(t[i]));
                }
            }
        }
#pragma unroll
        for (int d = 64 / GROUPS; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
        const int e = m > 0.0f && m < __builtin_inff() ? __builtin_amdgcn_frexp_expf(m) - 15 : 0;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = __builtin_ldexpf(v[s][i], -e);
                hi[s][i] = (_Float16)x;
                const float h = (float)hi[s][i];
                lo[s][i] = (_Float16)(__builtin_fabsf(h) < __builtin_inff() ? x - h : 0.0f);
            }
        return e;
    }

    // 16x16 blocks with four rows per lane (A's operand first): acc[tm][tn][r]
    // is row row0 + 16 tm + 4 (lane / 16) + r, column col0 + 16 tn + lane % 16.
    template <int TM, int TN>
    __device__ __forceinline__ void add16(v4f (&acc)[TM][TN], int row0, int col0, int M, int N) const {
        const int lane = threadIdx.x & 63, j16 = lane & 15, g = lane >> 4;
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
            const int row = row0 + 16 * tm + j16;
            const int mine = adapter_of(row, M);
            uint32_t todo = (uint32_t)__builtin_amdgcn_ballot_w64(mine >= 0) & 0xFFFFu;
            if (!todo) continue;
            const float* lrow = low + (int64_t)min(row, M - 1) * rank_p;
            for (int p0 = 0; p0 < rank_p; p0 += 64) {
                v8h hi[2], lo[2];
                const int e = split_piece<2, 4>(lrow, p0, g, hi, lo);
                for (uint32_t left = todo; left;) {
                    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
                    const uint32_t rows = (uint32_t)__builtin_amdgcn_ballot_w64(mine == a) & 0xFFFFu;
                    left &= ~rows;
#pragma unroll
                    for (int tn = 0; tn < TN; ++tn) {
                        const int col = min(col0 + 16 * tn + j16, N - 1);
                        v4f sum = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            if (p0 + 32 * s >= rank_p) break;
                            const v8h b = lb_chunk(a, col, p0 + 8 * (4 * s + g), N);
                            sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi[s], b, sum, 0, 0, 0);
                            sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo[s], b, sum, 0, 0, 0);
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int er = __shfl(e, 4 * g + r);   // the exponent of row 4 g + r
                            if ((rows >> (4 * g + r)) & 1) acc[tm][tn][r] += __builtin_ldexpf(sum[r], er);
                        }
                    }
                }
            }
        }
    }

    // 32x32 blocks with one row per lane (LB's operand first): acc[i][j] holds
    // row row0 + 32 i + lane % 32, columns col0 + 32 j + 8 q + 4 (lane / 32) + e
    // in value 4 q + e.
    template <int MI>
    __device__ __forceinline__ void add32(v16f (&acc)[MI][2], int row0, int col0, int M, int N) const {
        const int lane = threadIdx.x & 63, lr = lane & 31, h = lane >> 5;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int row = row0 + 32 * i + lr;
            const int mine = adapter_of(row, M);
            const uint32_t todo = (uint32_t)__builtin_amdgcn_ballot_w64(mine >= 0);
            if (!todo) continue;
            const float* lrow = low + (int64_t)min(row, M - 1) * rank_p;
            for (int p0 = 0; p0 < rank_p; p0 += 64) {
                v8h hi[4], lo[4];
                const int e = split_piece<4, 2>(lrow, p0, h, hi, lo);
                for (uint32_t left = todo; left;) {
                    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
                    left &= ~(uint32_t)__builtin_amdgcn_ballot_w64(mine == a);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int col = min(col0 + 32 * j + lr, N - 1);
                        v16f sum;
#pragma unroll
                        for (int r = 0; r < 16; ++r) sum[r] = 0.0f;
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            if (p0 + 16 * s >= rank_p) break;
                            const v8h b = lb_chunk(a, col, p0 + 8 * (2 * s + h), N);
                            sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, hi[s], sum, 0, 0, 0);
                            sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, lo[s], sum, 0, 0, 0);
                        }
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (mine == a) acc[i][j][r] += __builtin_ldexpf(sum[r], e);
                    }
                }
            }
        }
    }

    // Four neighbouring columns of one row, on the vector units: for few rows,
    // where each usually has its own adapter and a block has nothing to share.
    __device__ __forceinline__ void add_row4(v4f& y, int row, int col, int M, int N) const {
        const int a = adapter_of(row, M);
        if (a < 0) return;
        const float* lrow = low + (int64_t)row * rank_p;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
        for (int r0 = 0; r0 < rank_p; r0 += 8) {
            const v4f l0 = *reinterpret_cast<const v4f*>(lrow + r0), l1 = *reinterpret_cast<const v4f*>(lrow + r0 + 4);
            v8h b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = lb_chunk(a, min(col + e, N - 1), r0, N);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[e] = __builtin_fmaf(i < 4 ? l0[i & 3] : l1[i & 3], (float)b[e][i], sum[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += sum[e];
    }
};

}  // namespace libgemm
