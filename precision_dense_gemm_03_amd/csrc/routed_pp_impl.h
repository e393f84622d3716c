// The ping-pong tile kernel (gemm_pp_impl.h) over row groups, and with the
// low-rank term of per-row adapters.
//
// Grouped: tiles of BM x 256, and with TAILS a group's last rows at the
// smallest of 64, 128, 192 and 256 rows that holds them (the four bodies share
// the LDS rings; pairs with E5M2 are built at 192 rows only, without TAILS). One
// workgroup per tile the host cannot rule out, and more (most_workgroups); one
// without a tile ends after its look at the offsets. A fixed number of workgroups
// walking the tiles measured slower: the walk's state cost the main loop its
// registers (47 spilled per lane with 256 rows).
#pragma once

#include "gemm_pp_impl.h"
#include "lora_extra.h"
#include "row_groups.h"

namespace libgemm {
namespace routed {

template <int ES, int OUT, int FA, int FB, bool BT, int BM, bool TAILS, bool LINES = false>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void grouped_pp_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, void* __restrict__ C,
    const int32_t* __restrict__ offsets, int groups, int rows, int N, int K, const float* __restrict__ sA,
    const float* __restrict__ sB, const float* __restrict__ sOut, int tiles_n, int eflags, int vec_out) {
    using T = pp::Pp<ES, BM>;
    LIBGEMM_PP_LDS(T);
    const RowTile t = find_row_tile<BM>(offsets, groups, rows, (int)wide_block(), tiles_n);
    if (t.m0 >= t.end) return;
    const int n0 = t.tn * T::BN;
    if (t.group < 0) {
        zero_rows<BM, T::BN, OUT == OUT_F32 ? 4 : (OUT == OUT_F16 ? 2 : 1)>(C, t.m0, t.end, n0, N);
        return;
    }
    const bool chan = (eflags & EPI_CHANNEL) != 0;
    const float* sb = sB ? sB + (chan ? (int64_t)t.group * N : t.group) : nullptr;
    const uint8_t* b = B + (int64_t)t.group * N * K * ES;
    const int left = t.end - t.m0;
    if constexpr (TAILS && BM > 64) {
        if (left <= 64) {
            pp::pp_body<ES, OUT, FA, FB, BT, false, 64, true, pp::NoExtra, LINES>(A, b, C, t.end, N, K, sA, sb, sOut, t.m0, n0, eflags,
                                                              vec_out, lds);
            return;
        }
    }
    if constexpr (TAILS && BM > 128) {
        if (left <= 128) {
            pp::pp_body<ES, OUT, FA, FB, BT, false, 128, true, pp::NoExtra, LINES>(A, b, C, t.end, N, K, sA, sb, sOut, t.m0, n0, eflags,
                                                               vec_out, lds);
            return;
        }
    }
    if constexpr (TAILS && BM > 192) {
        if (left <= 192) {
            pp::pp_body<ES, OUT, FA, FB, BT, false, 192, true, pp::NoExtra, LINES>(A, b, C, t.end, N, K, sA, sb, sOut, t.m0, n0, eflags,
                                                               vec_out, lds);
            return;
        }
    }
    pp::pp_body<ES, OUT, FA, FB, BT, false, BM, true, pp::NoExtra, LINES>(A, b, C, t.end, N, K, sA, sb, sOut, t.m0, n0, eflags, vec_out,
                                                      lds);
}

// FP16 rows of whole 128-byte lines: then the results go past the caches, whose
// room the operands keep (8192 x 4096 x 4096 in 8 groups, us: FP8 139 -> 125,
// FP16 280 -> 267).
inline bool whole_lines(const GemmArgs& a) { return ((uintptr_t)a.C & 127) == 0 && a.N % 64 == 0; }

// What the ping-pong kernel needs (pp_fits), and a grid that can be launched.
template <int ES>
bool grouped_pp_fits(const GroupedArgs& a) {
    const bool fits = a.b_kmajor ? pp::pp_fits<ES, true, 256>(a) : pp::pp_fits<ES, false, 256>(a);
    return fits && most_workgroups(a.M, a.groups, 128, (a.N + 255) / 256) <= kMostWorkgroups;
}

template <int ES, int FA, int FB, bool BT, int BM, bool TAILS = true>
hipError_t launch_grouped_pp(const GroupedArgs& a) {
    using T = pp::Pp<ES, BM>;
    const int64_t tiles_n = (a.N + T::BN - 1) / T::BN;
    const dim3 grid = wide_grid(most_workgroups(a.M, a.groups, BM, tiles_n));
    const int eflags = (a.out_dtype == OUT_E5M2 ? EPI_E5M2 : 0) | (a.channel ? EPI_CHANNEL : 0);
    const int64_t out_es = a.out_dtype == OUT_F32 ? 4 : (a.out_dtype == OUT_F16 ? 2 : 1);
    const int vec_out = pp::aligned16(a.C) && (a.N * out_es) % 16 == 0;
    const uint8_t* A = reinterpret_cast<const uint8_t*>(a.A);
    const uint8_t* B = reinterpret_cast<const uint8_t*>(a.B);
#define LIBGEMM_GO(OUT, LINES)                                                                                \
    grouped_pp_kernel<ES, OUT, FA, FB, BT, BM, TAILS, LINES><<<grid, T::NT, 0, a.stream>>>(                          \
        A, B, a.C, a.offsets, (int)a.groups, (int)a.M, (int)a.N, (int)a.K, a.sA, a.sB, a.sOut, (int)tiles_n,  \
        eflags, vec_out)
    if (a.out_dtype == OUT_F32) {
        LIBGEMM_GO(OUT_F32, false);
    } else if (a.out_dtype == OUT_F16) {
        if (whole_lines(a)) LIBGEMM_GO(OUT_F16, true);
        else LIBGEMM_GO(OUT_F16, false);
    } else if constexpr (ES == 1) {
        LIBGEMM_GO(OUT_E4M3, false);
    } else {
        return hipErrorInvalidValue;
    }
#undef LIBGEMM_GO
    return hipGetLastError();
}

template <int ES, int OUT, int FA, int FB, int BM, bool LINES>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void lora_pp_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, void* __restrict__ C, int M, int N, int K,
    const float* __restrict__ sA, const float* __restrict__ sB, int tiles_m, int tiles_n, int eflags, int vec_out,
    LoraExtra ext) {
    using T = pp::Pp<ES, BM>;
    LIBGEMM_PP_LDS(T);
    if (past_last_block((int64_t)tiles_m * tiles_n)) return;
    int tm, tn;
    tile_coords((int)wide_block(), tiles_m, tiles_n, tm, tn);
    pp::pp_body<ES, OUT, FA, FB, true, false, BM, true, LoraExtra, LINES>(A, B, C, M, N, K, sA, sB, nullptr, tm * BM,
                                                                         tn * 256, eflags, vec_out, lds, ext);
}

template <int ES, int FA, int FB, int BM>
hipError_t launch_lora_pp(const LoraArgs& a) {
    const int64_t tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + 255) / 256;
    if (tiles_m * tiles_n > kMostWorkgroups) return hipErrorInvalidValue;
    const dim3 grid = wide_grid(tiles_m * tiles_n);
    const int eflags = a.channel ? EPI_CHANNEL : 0;
    const int vec_out = pp::aligned16(a.C) && (a.N * (a.out_dtype == OUT_F32 ? 4 : 2)) % 16 == 0;
    const uint8_t* A = reinterpret_cast<const uint8_t*>(a.A);
    const uint8_t* B = reinterpret_cast<const uint8_t*>(a.B);
    const LoraExtra ext{a.low, a.adapter, reinterpret_cast<const _Float16*>(a.LB), (int)a.rank,
                        (int)((a.rank + 7) / 8 * 8), (int)a.adapters, a.low_slices, a.M * ((a.rank + 7) / 8 * 8)};
#define LIBGEMM_GO(OUT, LINES)                                                                                  \
    lora_pp_kernel<ES, OUT, FA, FB, BM, LINES><<<grid, 512, 0, a.stream>>>(                                     \
        A, B, a.C, (int)a.M, (int)a.N, (int)a.K, a.sA, a.sB, (int)tiles_m, (int)tiles_n, eflags, vec_out, ext)
    if (a.out_dtype == OUT_F32) LIBGEMM_GO(OUT_F32, false);
    else if (a.out_dtype != OUT_F16) return hipErrorInvalidValue;
    else if (whole_lines(a)) LIBGEMM_GO(OUT_F16, true);
    else LIBGEMM_GO(OUT_F16, false);
#undef LIBGEMM_GO
    return hipGetLastError();
}

}  // namespace routed
}  // namespace libgemm
