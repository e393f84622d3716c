// Gradient to the weights where one operand was kept as 8-bit values with scales
// (row_io.h): C[g] = A[rows of g]^T B[rows of g] with A or B such an operand, the
// kernels of gemm_wgrad_impl.h.
#include "gemm_wgrad_impl.h"

namespace libgemm {

namespace {

template <int QS, int FMT>
hipError_t launch(const GroupedArgs& a, const uint8_t* scale) {
    const int pick = choose_wgrad(a, QS), size = pick == kSplit64 ? 64 : pick;
    const int64_t tiles_m = (a.M + size - 1) / size, tiles_n = (a.N + size - 1) / size;
    const int64_t blocks = wgrad_blocks(a.groups, tiles_m, tiles_n);
    if (blocks > kMostWorkgroups) return hipErrorInvalidValue;
    const dim3 grid = wide_grid(blocks);
    const int rows = (int)a.K, M = (int)a.M, N = (int)a.N, groups = (int)a.groups;
    const bool lines = ((uintptr_t)a.C & 127) == 0 && a.N * (a.out_dtype == OUT_F32 ? 4 : 2) % 128 == 0;
    const int vec_out = pp::aligned16(a.C);
    const MxOperand mx{scale, ((QS == 1 ? a.M : a.N) + kMxBlock - 1) / kMxBlock};
#define LIBGEMM_PP(OUT, LINES)                                                                             \
    wgrad_pp_kernel<OUT, LINES, QS, FMT><<<grid, 512, 0, a.stream>>>(                                       \
        (const uint8_t*)a.A, (const uint8_t*)a.B, a.C, a.offsets, groups, rows, M, N, (int)tiles_m,        \
        (int)tiles_n, vec_out, mx)
#define LIBGEMM_CUT(OUT, TS, KG, CUT)                                                                 \
    wgrad_tile_kernel<OUT, TS, CUT, QS, FMT, KG><<<grid, 256 * KG, 0, a.stream>>>(                    \
        (const _Float16*)a.A, (const _Float16*)a.B, a.C, a.offsets, groups, rows, M, N, (int)tiles_m, \
        (int)tiles_n, mx)
#define LIBGEMM_TILE(OUT, TS, KG)                                                                     \
    do {                                                                                              \
        if (M % 8 || N % 8) LIBGEMM_CUT(OUT, TS, KG, true);                                           \
        else LIBGEMM_CUT(OUT, TS, KG, false);                                                         \
    } while (0)
    const bool f32 = a.out_dtype == OUT_F32;
    if (size == 256) {
        if (f32 && lines) LIBGEMM_PP(OUT_F32, true);
        else if (f32) LIBGEMM_PP(OUT_F32, false);
        else if (lines) LIBGEMM_PP(OUT_F16, true);
        else LIBGEMM_PP(OUT_F16, false);
    } else if (size == 128) {
        if (f32) LIBGEMM_TILE(OUT_F32, 128, 1);
        else LIBGEMM_TILE(OUT_F16, 128, 1);
    } else if (pick == 64) {
        if (f32) LIBGEMM_TILE(OUT_F32, 64, 1);
        else LIBGEMM_TILE(OUT_F16, 64, 1);
    } else {
        if (f32) LIBGEMM_TILE(OUT_F32, 64, 4);
        else LIBGEMM_TILE(OUT_F16, 64, 4);
    }
#undef LIBGEMM_PP
#undef LIBGEMM_TILE
#undef LIBGEMM_CUT
    return hipGetLastError();
}

}  // namespace

const char* wgrad_mx_kernel_name(const GroupedArgs& a, int qs) {
    switch (choose_wgrad(a, qs)) {
        case 256: return "wgrad_pp";
        case 128: return "wgrad_tile_128";
        case 64: return "wgrad_tile_64";
        default: return "wgrad_tile_64_split";
    }
}

hipError_t launch_wgrad_mx(const GroupedArgs& a, const uint8_t* scale, int fmt, int qs) {
    if (a.M <= 0 || a.N <= 0 || a.groups <= 0) return hipSuccess;
    if (qs == 1) return fmt == FMT_E5M2 ? launch<1, FMT_E5M2>(a, scale) : launch<1, FMT_E4M3>(a, scale);
    return fmt == FMT_E5M2 ? launch<2, FMT_E5M2>(a, scale) : launch<2, FMT_E4M3>(a, scale);
}

}  // namespace libgemm
