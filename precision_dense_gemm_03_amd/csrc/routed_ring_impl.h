// The deep-ring kernel (gemm_ring_impl.h) over row groups of a few rows, and
// with the low-rank term of per-row adapters.
//
// Grouped: the weights stream once and bound the call, so what counts is loads
// in flight per compute unit. Tiles are 64 rows x 64 columns; a tile with up to
// 16 or 32 rows runs at that height, and the three bodies share an LDS ring
// of 72 KiB (7, 6 or 4 stages), so that two workgroups fit a compute unit and
// one's first loads run under the other's stream. 16 rows in 16 groups of
// 4096 x 4096 FP16 weights: 68.9 us, 5.85 TB/s of the weights in use; tiles of
// 32 columns, three workgroups per unit: 87.4 us.
#pragma once

#include "gemm_ring_impl.h"
#include "lora_extra.h"
#include "row_groups.h"

namespace libgemm {
namespace routed {

constexpr int kRingBytes = 72 * 1024;

template <int ES, int OUT, int FA, int FB, bool BT>
__global__ __launch_bounds__(256) void grouped_ring_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, void* __restrict__ C,
    const int32_t* __restrict__ offsets, int groups, int rows, int N, int K, const float* __restrict__ sA,
    const float* __restrict__ sB, const float* __restrict__ sOut, int tiles_n, int eflags, int vec_out) {
    constexpr int BN = 64;
    constexpr int S16 = kRingBytes / ((16 + BN) * 128), S32 = kRingBytes / ((32 + BN) * 128);
    constexpr int S64 = kRingBytes / ((64 + BN) * 128);
    __shared__ __attribute__((aligned(1024))) uint8_t ring[kRingBytes];
    __shared__ v4f red[ring::Ring<ES, 16, BN, BT, S16>::RED_SLOTS];
    const RowTile t = find_row_tile<64>(offsets, groups, rows, (int)wide_block(), tiles_n);
    if (t.m0 >= t.end) return;
    const int n0 = t.tn * BN;
    if (t.group < 0) {
        zero_rows<64, BN, OUT == OUT_F32 ? 4 : (OUT == OUT_F16 ? 2 : 1)>(C, t.m0, t.end, n0, N);
        return;
    }
    const bool chan = (eflags & EPI_CHANNEL) != 0;
    const float* sb = sB ? sB + (chan ? (int64_t)t.group * N : t.group) : nullptr;
    const uint8_t* b = B + (int64_t)t.group * N * K * ES;
    if (t.end - t.m0 <= 16)
        ring::ring_body<ES, 16, BN, OUT, FA, FB, BT, S16, true>(A, b, C, t.end, N, K, sA, sb, sOut, t.m0, n0, eflags,
                                                                vec_out, ring, red);
    else if (t.end - t.m0 <= 32)
        ring::ring_body<ES, 32, BN, OUT, FA, FB, BT, S32, true>(A, b, C, t.end, N, K, sA, sb, sOut, t.m0, n0, eflags,
                                                                vec_out, ring, red);
    else
        ring::ring_body<ES, 64, BN, OUT, FA, FB, BT, S64, true>(A, b, C, t.end, N, K, sA, sb, sOut, t.m0, n0, eflags,
                                                                vec_out, ring, red);
}

template <int ES>
bool grouped_ring_fits(const GroupedArgs& a) {
    const bool fits = a.b_kmajor ? ring::ring_fits<ES, 64, true>(a, 64) : ring::ring_fits<ES, 64, false>(a, 64);
    return fits && most_workgroups(a.M, a.groups, 64, (a.N + 63) / 64) <= kMostWorkgroups;
}

template <int ES, int FA, int FB, bool BT>
hipError_t launch_grouped_ring(const GroupedArgs& a) {
    const int64_t tiles_n = (a.N + 63) / 64;
    const dim3 grid = wide_grid(most_workgroups(a.M, a.groups, 64, tiles_n));
    const int eflags = (a.out_dtype == OUT_E5M2 ? EPI_E5M2 : 0) | (a.channel ? EPI_CHANNEL : 0);
    const int64_t out_es = a.out_dtype == OUT_F32 ? 4 : (a.out_dtype == OUT_F16 ? 2 : 1);
    const int vec_out = ((uintptr_t)a.C % (4 * out_es)) == 0 && (a.N % 4) == 0;
    const uint8_t* A = reinterpret_cast<const uint8_t*>(a.A);
    const uint8_t* B = reinterpret_cast<const uint8_t*>(a.B);
#define LIBGEMM_GO(OUT)                                                                                         \
    grouped_ring_kernel<ES, OUT, FA, FB, BT><<<grid, 256, 0, a.stream>>>(                                   \
        A, B, a.C, a.offsets, (int)a.groups, (int)a.M, (int)a.N, (int)a.K, a.sA, a.sB, a.sOut, (int)tiles_n,    \
        eflags, vec_out)
    if (a.out_dtype == OUT_F32) {
        LIBGEMM_GO(OUT_F32);
    } else if (a.out_dtype == OUT_F16) {
        LIBGEMM_GO(OUT_F16);
    } else if constexpr (ES == 1) {
        LIBGEMM_GO(OUT_E4M3);
    } else {
        return hipErrorInvalidValue;
    }
#undef LIBGEMM_GO
    return hipGetLastError();
}

// The adapters' ring: K tiles per barrier and stages. 16 rows, N = K = 4096,
// rank 16, cold weight: 14.8 us with 4 tiles of 16 x 16 per barrier and 12
// stages (8: 14.3, but 64 rows 22.1 against 21.6), 20.6 with one and 8 (any
// depth up to 32 stages then 20.6 to 25.7). Wider tiles: 128 rows 32.9 us with
// 2, 36.2 with 4.
template <int BM, int BN>
struct LoraRing {
    static constexpr int P = BM * BN <= 512 ? 4 : 2;
    static constexpr int FIT = 128 * 1024 / ((BM + BN) * 128), S = (FIT < 12 ? FIT : 12) / P * P;
};

template <int ES, int BM, int BN, int OUT, int FA, int FB>
__global__ __launch_bounds__(256) void lora_ring_kernel(const uint8_t* __restrict__ A, const uint8_t* __restrict__ B,
                                                        void* __restrict__ C, int M, int N, int K,
                                                        const float* __restrict__ sA, const float* __restrict__ sB,
                                                        int tiles_m, int tiles_n, int eflags, int vec_out,
                                                        LoraExtra ext) {
    constexpr int S = LoraRing<BM, BN>::S, P = LoraRing<BM, BN>::P;
    using T = ring::Ring<ES, BM, BN, true, S>;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[T::S * T::STAGE];
    __shared__ v4f red[T::RED_SLOTS];
    if (past_last_block((int64_t)tiles_m * tiles_n)) return;
    int tm, tn;
    tile_coords((int)wide_block(), tiles_m, tiles_n, tm, tn);
    ring::ring_body<ES, BM, BN, OUT, FA, FB, true, S, true, LoraExtra, P>(A, B, C, M, N, K, sA, sB, nullptr, tm * BM,
                                                                      tn * BN, eflags, vec_out, ring, red, ext);
}

template <int ES, int FA, int FB, int BM, int BN>
hipError_t launch_lora_ring(const LoraArgs& a) {
    const int64_t tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN;
    if (tiles_m * tiles_n > kMostWorkgroups) return hipErrorInvalidValue;
    const dim3 grid = wide_grid(tiles_m * tiles_n);
    const int eflags = a.channel ? EPI_CHANNEL : 0;
    const int vec_out = ((uintptr_t)a.C % (a.out_dtype == OUT_F32 ? 16 : 8)) == 0 && (a.N % 4) == 0;
    const uint8_t* A = reinterpret_cast<const uint8_t*>(a.A);
    const uint8_t* B = reinterpret_cast<const uint8_t*>(a.B);
    const LoraExtra ext{a.low, a.adapter, reinterpret_cast<const _Float16*>(a.LB), (int)a.rank,
                        (int)((a.rank + 7) / 8 * 8), (int)a.adapters, a.low_slices, a.M * ((a.rank + 7) / 8 * 8)};
    if (a.out_dtype == OUT_F32)
        lora_ring_kernel<ES, BM, BN, OUT_F32, FA, FB><<<grid, 256, 0, a.stream>>>(
            A, B, a.C, (int)a.M, (int)a.N, (int)a.K, a.sA, a.sB, (int)tiles_m, (int)tiles_n, eflags, vec_out, ext);
    else if (a.out_dtype == OUT_F16)
        lora_ring_kernel<ES, BM, BN, OUT_F16, FA, FB><<<grid, 256, 0, a.stream>>>(
            A, B, a.C, (int)a.M, (int)a.N, (int)a.K, a.sA, a.sB, (int)tiles_m, (int)tiles_n, eflags, vec_out, ext);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

template <int ES, int FA, int FB>
hipError_t launch_lora_ring_any(const LoraArgs& a) {
    static hipError_t (*const launch[])(const LoraArgs&) = {
        launch_lora_ring<ES, FA, FB, 16, 16>, launch_lora_ring<ES, FA, FB, 16, 32>, launch_lora_ring<ES, FA, FB, 16, 64>,
        launch_lora_ring<ES, FA, FB, 32, 32>, launch_lora_ring<ES, FA, FB, 32, 64>, launch_lora_ring<ES, FA, FB, 64, 64>};
    int64_t cost = 0;
    return launch[lora_ring_shape(a.M, a.N, &cost)](a);   // in kLoraRingShapes' order
}

}  // namespace routed
}  // namespace libgemm
