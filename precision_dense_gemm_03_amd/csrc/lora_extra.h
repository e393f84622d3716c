// The low-rank term of a product with per-row adapters, added to a tile's
// accumulators after its K loop (lora.hip computes the low-rank values):
//
//   y[i, j] = base[i, j] + sum_r low[i, r] LB[a_i, j, r],   a_i the row's adapter
//
// low is FP32 and LB FP16. The tile kernels (add16, add_tile) split each row's
// low values into two FP16 numbers, hi + lo, after scaling the row's piece of 64
// by a power of two that puts its largest value into [2^14, 2^15) (an infinity
// counts as 2^127). hi is off by at most 2^-11 of the value and lo by at most
// 2^-11 of what hi left, or half FP16's smallest step, so a value enters to 2^-22
// of itself or 2^-39 of the piece's largest, whichever is more: two bits fewer
// than FP32 holds. That is the choice made here: K products summed in FP32 are
// seldom that exact, and a third part would cost half as many matrix
// instructions again. The deep-ring kernel (add_row4, few rows) multiplies the
// FP32 values as they are. The scaling is undone on the FP32 sum, exactly. Both
// halves meet LB's operand, loaded once.
//
// An infinity of LB must meet hi alone (lo may be zero, or of the other sign).
// add_tile looks for them as it stages LB; the tiles of add16 compute elements
// that came out as NaN again, one by one (repair16; looking at LB's values there,
// or at each sum, cost 6 to 17 % where rows of many adapters share a block).
//
// Rows of one block may have several adapters: each adapter present multiplies
// the whole block and only its rows take the sum, so no other adapter's values
// (NaN included) reach a row.
#pragma once

#include "device_common.h"

namespace libgemm {

// Top bit of each half that is an infinity or a NaN, in four words.
__device__ __forceinline__ v4u non_finite(v8h b) {
    v4u w = __builtin_bit_cast(v4u, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ((w[i] & 0x7FFF7FFFu) + 0x04000400u) & 0x80008000u;
    return w;
}

__device__ __forceinline__ bool any_non_finite(v8h b) {
    const v4u w = non_finite(b);
    return (w[0] | w[1] | w[2] | w[3]) != 0u;
}

// The finite halves, zero in the others' place.
__device__ __forceinline__ v8h finite_part(v8h b) {
    v4u w = __builtin_bit_cast(v4u, b);
    const v4u bad = non_finite(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] &= ~((bad[i] >> 15) * 0xFFFFu);
    return __builtin_bit_cast(v8h, w);
}

struct LoraExtra {
    static constexpr bool kActive = true, kStores = false, kFinish = false;
    const float* low;         // slices of [rows, rank_p], zero from rank on
    const int32_t* adapter;   // [rows]
    const _Float16* LB;       // [adapters, N, rank]
    int rank, rank_p;         // rank_p: rank rounded up to a multiple of 8
    int adapters;
    int slices;               // low is the sum of this many arrays, low_step values apart
    int64_t low_step;

    // Four of a row's low-rank values, the slices added in order.
    __device__ __forceinline__ v4f low4(const float* p) const {
        v4f v = *reinterpret_cast<const v4f*>(p);
        for (int s = 1; s < slices; ++s) v += *reinterpret_cast<const v4f*>(p + s * low_step);
        return v;
    }

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

    // STEPS chunks of 8 values of a row, from r0 on and `step` apart, as hi and
    // lo halves; the lanes lane ^ d, d = first_d, 2 first_d, .. below end_d, hold
    // the rest of the row's piece. Returns the piece's exponent.
    template <int STEPS>
    __device__ __forceinline__ int split_chunks(const float* row, int r0, int step, int first_d, int end_d,
                                                v8h (&hi)[STEPS], v8h (&lo)[STEPS]) const {
        float v[STEPS][8];
        float m = 0.0f;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int r = r0 + step * s;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4f t = v4f{0.f, 0.f, 0.f, 0.f};
                if (r < rank_p) t = low4(row + r + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[s][4 * h + i] = t[i];
                    m = fmaxf(m, __builtin_fabsf(t[i]));
                }
            }
        }
        for (int d = first_d; d < end_d; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
        // (beside an infinity the other values only have to stay finite)
        const int e = m > 0.0f ? (m < __builtin_inff() ? __builtin_amdgcn_frexp_expf(m) : 128) - 15 : 0;
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
                const int e = split_chunks<2>(lrow, p0 + 8 * g, 32, 16, 64, hi, lo);
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

    // After add16 and the stores: elements that came out as NaN, from LB's
    // infinity against lo or as the formula gives them, again in FP32, one by
    // one. product(row, col) gives the product alone, store(row, col, y) stores.
    template <int TM, int TN, class Product, class Store>
    __device__ __forceinline__ void repair16(const v4f (&acc)[TM][TN], int row0, int col0, int M, int N,
                                             Product product, Store store) const {
        bool nan = false;
#pragma unroll
        for (int i = 0; i < TM * TN; ++i)
            nan |= __builtin_isunordered(acc[i / TN][i % TN][0], acc[i / TN][i % TN][1]) |
                   __builtin_isunordered(acc[i / TN][i % TN][2], acc[i / TN][i % TN][3]);
        if (__builtin_expect(__builtin_amdgcn_ballot_w64(nan) == 0, 1)) return;
        const int lane = threadIdx.x & 63, j16 = lane & 15, g = lane >> 4;
        uint64_t todo = 0;
#pragma unroll
        for (int i = 0; i < 4 * TM * TN; ++i) {
            const float y = acc[i / 4 / TN][i / 4 % TN][i % 4];
            if (y != y) todo |= (uint64_t)1 << i;
        }
#pragma unroll 1
        for (; todo; todo &= todo - 1) {
            const int i = __builtin_ctzll(todo);
            const int row = row0 + 16 * (i / (4 * TN)) + 4 * g + i % 4, col = col0 + 16 * (i / 4 % TN) + j16;
            const int a = adapter_of(row, M);
            if (a >= 0 && col < N) store(row, col, product(row, col) + one_term(row, col, a, N));
        }
    }

    // One element of the term, in FP32.
    __device__ __forceinline__ float one_term(int row, int col, int a, int N) const {
        const float* l = low + (int64_t)row * rank_p;
        const _Float16* b = LB + ((int64_t)a * N + col) * rank;
        float sum = 0.0f;
#pragma unroll 1
        for (int r = 0; r < rank; ++r) {
            float v = l[r];
#pragma unroll 1
            for (int s = 1; s < slices; ++s) v += l[r + s * low_step];
            sum = __builtin_fmaf(v, (float)b[r], sum);
        }
        return sum;
    }

    // A 256-column tile of the ping-pong kernel (its acc, LDS regions and wave
    // layout: acc[i][j] holds row MR G + 32 i + lane % 32, columns 64 wj + 32 j +
    // 8 q + 4 (lane / 32) + e in value 4 q + e). After the K loop the LDS is
    // free: the tile's low-rank values go there split, once for all waves (hi
    // in region a[0], lo in a[1], 128 bytes of a row's piece each; the row's
    // exponent and adapter in a[2]), then for each adapter of the tile its 256
    // rows of LB (b[0], b[1]). So the wait for memory is one per adapter, and
    // the accumulators, which leave few registers, meet operands from LDS.
    // (Operands straight from memory, a wave for itself: 27 us of 137 for 4096
    // rows, N = K = 4096, rank 64.)
    template <int MI, class Lds>
    __device__ __forceinline__ void add_tile(v16f (&acc)[MI][2], const Lds& lds, int m0, int n0, int G, int wj, int M,
                                             int N) const {
        constexpr int BM = 64 * MI, MR = 32 * MI;
        const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, h = lane >> 5;
        LDS_AS int* ids = (LDS_AS int*)lds.a[2];
        LDS_AS int* exps = ids + BM;
        LDS_AS int* special = exps + BM;   // whether an infinity or NaN of LB was met
        auto slot = [](int r, int c) __attribute__((always_inline)) -> int {
            return r * 128 + ((c ^ ((r & 7) ^ ((r >> 3) & 1))) << 4);
        };
        const int srow = tid >> 1, half = tid & 1;   // staging: 32 values of a row (of low, of LB) per thread
        if (tid < BM) ids[tid] = adapter_of(m0 + tid, M);
        if (tid == 0) *special = 0;
        for (int p0 = 0; p0 < rank_p; p0 += 64) {
            if (srow < BM) {
                v8h hi[4], lo[4];
                const int e =
                    split_chunks<4>(low + (int64_t)min(m0 + srow, M - 1) * rank_p, p0 + 32 * half, 8, 1, 2, hi, lo);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    *(LDS_AS v8h*)(lds.a[0] + slot(srow, 4 * half + q)) = hi[q];
                    *(LDS_AS v8h*)(lds.a[1] + slot(srow, 4 * half + q)) = lo[q];
                }
                if (half == 0) exps[srow] = e;
            }
            __syncthreads();
            // the tile's adapters, one after another (every wave goes through the same list)
            int id[(BM + 63) / 64];
#pragma unroll
            for (int k = 0; k < (BM + 63) / 64; ++k) id[k] = ids[64 * k + lane];
            for (;;) {
                int a = -1;
#pragma unroll
                for (int k = 0; k < (BM + 63) / 64; ++k) {
                    const uint64_t some = __builtin_amdgcn_ballot_w64(id[k] >= 0);
                    if (a < 0 && some) a = __builtin_amdgcn_readlane(id[k], __builtin_ctzll(some));
                }
                if (a < 0) break;
#pragma unroll
                for (int k = 0; k < (BM + 63) / 64; ++k) id[k] = id[k] == a ? -1 : id[k];
                LDS_AS uint8_t* lb = srow < 128 ? lds.b[0] : lds.b[1];
                bool bad = false;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v8h v = lb_chunk(a, min(n0 + srow, N - 1), p0 + 32 * half + 8 * q, N);
                    bad |= any_non_finite(v);
                    *(LDS_AS v8h*)(lb + slot(srow & 127, 4 * half + q)) = v;
                }
                if (__builtin_amdgcn_ballot_w64(bad) != 0 && lane == 0) *special = 1;
                __syncthreads();
                const bool finite = *special == 0;
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const int r = MR * G + 32 * i + lr;
                    const bool mine = ids[r] == a;
                    if (__builtin_amdgcn_ballot_w64(mine) == 0) continue;
                    const int e = exps[r];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = 64 * (wj & 1) + 32 * j + lr;
                        const LDS_AS uint8_t* b = (wj < 2 ? lds.b[0] : lds.b[1]);
                        v16f sum;
#pragma unroll
                        for (int x = 0; x < 16; ++x) sum[x] = 0.0f;
                        for (int s = 0; s < 4 && p0 + 16 * s < rank_p; ++s) {
                            v8h bo = *(const LDS_AS v8h*)(b + slot(c, 2 * s + h));
                            const v8h ho = *(const LDS_AS v8h*)(lds.a[0] + slot(r, 2 * s + h));
                            const v8h lw = *(const LDS_AS v8h*)(lds.a[1] + slot(r, 2 * s + h));
                            sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(bo, ho, sum, 0, 0, 0);
                            if (!finite) bo = finite_part(bo);
                            sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(bo, lw, sum, 0, 0, 0);
                        }
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            if (mine) acc[i][j][x] += __builtin_ldexpf(sum[x], e);
                    }
                }
                __syncthreads();
            }
            __syncthreads();   // the next piece (or the stores' staging) overwrites the LDS
        }
    }

    // Few rows: each usually has its own adapter and a block has nothing to
    // share, so the term goes through the vector units, four neighbouring
    // columns of one row per lane, a row's low-rank values in pieces of 8 that
    // the waves holding the block's partial sums share out (wave group kg of KW
    // takes pieces kg, kg + KW, ...). A lane's first piece is fetched before
    // the K loop, whose length hides LB's way from memory.
    struct Piece {
        int adapter;
        v4f l[2];
        v8h b[4];
    };

    __device__ __forceinline__ void fetch(Piece& p, int row, int col, int r0, int N) const {
        const float* lrow = low + (int64_t)row * rank_p + r0;
        p.l[0] = low4(lrow);
        p.l[1] = low4(lrow + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) p.b[e] = lb_chunk(p.adapter, min(col + e, N - 1), r0, N);
    }

    __device__ __forceinline__ void prefetch(Piece& p, int row, int col, int kg, int M, int N) const {
        p.adapter = adapter_of(row, M);
        if (p.adapter >= 0 && 8 * kg < rank_p) fetch(p, row, col, 8 * kg, N);
    }

    __device__ __forceinline__ void add_row4(v4f& y, Piece& p, int row, int col, int kg, int KW, int N) const {
        if (p.adapter < 0 || 8 * kg >= rank_p) return;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int r0 = 8 * kg;;) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum[e] = __builtin_fmaf(p.l[i >> 2][i & 3], (float)p.b[e][i], sum[e]);
            r0 += 8 * KW;
            if (r0 >= rank_p) break;
            fetch(p, row, col, r0, N);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += sum[e];
    }
};

}  // namespace libgemm
