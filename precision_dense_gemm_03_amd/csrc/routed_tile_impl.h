// The register-staged tile kernel for products whose weight depends on the
// row: over row groups, and with the low-rank term of per-row adapters. Its
// tile body (gemm_tile_impl.h) takes operands of any alignment here, so these
// kernels serve every size; the faster kernels take what their alignment and
// shape rules allow (routed.cpp).
//
// Grouped: a fixed number of workgroups walks the tiles (row_groups.h), so
// that the bound on the tiles the host has to launch for, up to one more row
// tile per group than there are, costs no empty workgroups.
#pragma once

#include "gemm_tile_impl.h"
#include "lora_extra.h"
#include "row_groups.h"

namespace libgemm {
namespace routed {

constexpr int kTileWorkgroups = 256 * 4;   // 4 of 64 x 64 fit a compute unit's LDS

template <int ES, int OUT, int BM, int BK, int FA, int FB, bool BT>
__global__ __launch_bounds__(256) void grouped_tile_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, void* __restrict__ C,
    const int32_t* __restrict__ offsets, int groups, int rows, int N, int K, const float* __restrict__ sA,
    const float* __restrict__ sB, const float* __restrict__ sOut, int most, int tiles_n, int eflags) {
    constexpr int BN = BM;
    const bool chan = (eflags & EPI_CHANNEL) != 0;
    for (int id = blockIdx.x; id < most; id += gridDim.x) {   // the grid is a multiple of 8: one XCD's tiles
        const RowTile t = find_row_tile<BM>(offsets, groups, rows, id, tiles_n);
        if (t.m0 >= t.end) break;
        const int tn = t.tn;
        if (t.group < 0) {
            zero_rows<BM, BN, OUT == OUT_F32 ? 4 : (OUT == OUT_F16 ? 2 : 1)>(C, t.m0, t.end, tn * BN, N);
            continue;
        }
        const float* sb = sB ? sB + (chan ? (int64_t)t.group * N : t.group) : nullptr;
        tile::tile_body<ES, OUT, BM, BN, BK, 2, 2, FA, FB, BT, ES, true>(A, B + (int64_t)t.group * N * K * ES, C, t.end, N, K,
                                                                  sA, sb, sOut, t.m0, tn * BN, 1, eflags, K, 0);
    }
}

template <int ES, int BM, int FA, int FB, bool BT>
hipError_t launch_grouped_tile(const GroupedArgs& a) {
    constexpr int BK = 128 / ES;
    const int64_t tiles_n = (a.N + BM - 1) / BM, most = most_workgroups(a.M, a.groups, BM, tiles_n);
    if (most > 0x7FFFFFFF - kTileWorkgroups) return hipErrorInvalidValue;
    const unsigned grid = (unsigned)(most < kTileWorkgroups ? most : kTileWorkgroups);
    const int eflags = (a.out_dtype == OUT_E5M2 ? EPI_E5M2 : 0) | (a.channel ? EPI_CHANNEL : 0);
    const uint8_t* A = reinterpret_cast<const uint8_t*>(a.A);
    const uint8_t* B = reinterpret_cast<const uint8_t*>(a.B);
#define LIBGEMM_GO(OUT)                                                                                         \
    grouped_tile_kernel<ES, OUT, BM, BK, FA, FB, BT><<<grid, 256, 0, a.stream>>>(                               \
        A, B, a.C, a.offsets, (int)a.groups, (int)a.M, (int)a.N, (int)a.K, a.sA, a.sB, a.sOut, (int)most,       \
        (int)tiles_n, eflags)
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

template <int ES, int OUT, int BM, int BK, int FA, int FB>
__global__ __launch_bounds__(256) void lora_tile_kernel(const uint8_t* __restrict__ A, const uint8_t* __restrict__ B,
                                                        void* __restrict__ C, int M, int N, int K,
                                                        const float* __restrict__ sA, const float* __restrict__ sB,
                                                        int tiles_m, int tiles_n, int eflags, LoraExtra ext) {
    if (past_last_block((int64_t)tiles_m * tiles_n)) return;
    int tm, tn;
    tile_coords((int)wide_block(), tiles_m, tiles_n, tm, tn);
    tile::tile_body<ES, OUT, BM, BM, BK, 2, 2, FA, FB, true, ES, true, LoraExtra>(A, B, C, M, N, K, sA, sB, nullptr, tm * BM,
                                                                           tn * BM, 1, eflags, K, 0, ext);
}

inline LoraExtra extra_of(const LoraArgs& a) {
    return LoraExtra{a.low, a.adapter, reinterpret_cast<const _Float16*>(a.LB), (int)a.rank,
                     (int)((a.rank + 7) / 8 * 8), (int)a.adapters, a.low_slices, a.M * ((a.rank + 7) / 8 * 8)};
}

template <int ES, int BM, int FA, int FB>
hipError_t launch_lora_tile(const LoraArgs& a) {
    constexpr int BK = 128 / ES;
    const int64_t tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BM - 1) / BM;
    if (tiles_m * tiles_n > kMostWorkgroups) return hipErrorInvalidValue;
    const dim3 grid = wide_grid(tiles_m * tiles_n);
    const int eflags = a.channel ? EPI_CHANNEL : 0;
    const uint8_t* A = reinterpret_cast<const uint8_t*>(a.A);
    const uint8_t* B = reinterpret_cast<const uint8_t*>(a.B);
    if (a.out_dtype == OUT_F32)
        lora_tile_kernel<ES, OUT_F32, BM, BK, FA, FB><<<grid, 256, 0, a.stream>>>(
            A, B, a.C, (int)a.M, (int)a.N, (int)a.K, a.sA, a.sB, (int)tiles_m, (int)tiles_n, eflags, extra_of(a));
    else if (a.out_dtype == OUT_F16)
        lora_tile_kernel<ES, OUT_F16, BM, BK, FA, FB><<<grid, 256, 0, a.stream>>>(
            A, B, a.C, (int)a.M, (int)a.N, (int)a.K, a.sA, a.sB, (int)tiles_m, (int)tiles_n, eflags, extra_of(a));
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

// Operand-format dispatch.
template <int BM, bool BT>
hipError_t grouped_tile_fp8(const GroupedArgs& a) {
    switch (a.fmt_a * 2 + a.fmt_b) {
        case 0: return launch_grouped_tile<1, BM, 0, 0, BT>(a);
        case 1: return launch_grouped_tile<1, BM, 0, 1, BT>(a);
        case 2: return launch_grouped_tile<1, BM, 1, 0, BT>(a);
        default: return launch_grouped_tile<1, BM, 1, 1, BT>(a);
    }
}

template <int BM>
hipError_t lora_tile_fp8(const LoraArgs& a) {
    switch (a.fmt_a * 2 + a.fmt_b) {
        case 0: return launch_lora_tile<1, BM, 0, 0>(a);
        case 1: return launch_lora_tile<1, BM, 0, 1>(a);
        case 2: return launch_lora_tile<1, BM, 1, 0>(a);
        default: return launch_lora_tile<1, BM, 1, 1>(a);
    }
}

}  // namespace routed
}  // namespace libgemm
