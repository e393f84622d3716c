// Gradient to the weights of products grouped by rows, FP16 operands (gemm_wgrad_impl.h).
#include "gemm_wgrad_impl.h"

namespace libgemm {

const char* wgrad_kernel_name(const GroupedArgs& a) {
    const int size = choose_wgrad(a);
    return size == 256 ? "wgrad_pp" : (size == 128 ? "wgrad_tile_128" : "wgrad_tile_64");
}

hipError_t launch_grouped_wgrad(const GroupedArgs& a) {
    if (a.M <= 0 || a.N <= 0 || a.groups <= 0) return hipSuccess;
    const int size = choose_wgrad(a);
    const int64_t tiles_m = (a.M + size - 1) / size, tiles_n = (a.N + size - 1) / size;
    const int64_t blocks = wgrad_blocks(a.groups, tiles_m, tiles_n);
    if (blocks > kMostWorkgroups) return hipErrorInvalidValue;
    const dim3 grid = wide_grid(blocks);
    const int rows = (int)a.K, M = (int)a.M, N = (int)a.N, groups = (int)a.groups;
    // Whole lines past the caches: 4096 rows, 8 groups, 2048 x 4096 FP16 102 -> 89
    // us; lines written in two parts, 18 groups of 2232 x 824: 17.9 -> 31.2.
    const bool lines = ((uintptr_t)a.C & 127) == 0 && a.N * (a.out_dtype == OUT_F32 ? 4 : 2) % 128 == 0;
    const int vec_out = pp::aligned16(a.C);
#define LIBGEMM_PP(OUT, LINES)                                                                             \
    wgrad_pp_kernel<OUT, LINES><<<grid, 512, 0, a.stream>>>(                                                \
        (const uint8_t*)a.A, (const uint8_t*)a.B, a.C, a.offsets, groups, rows, M, N, (int)tiles_m,        \
        (int)tiles_n, vec_out, MxOperand{})
#define LIBGEMM_CUT(OUT, TS, CUT)                                                                     \
    wgrad_tile_kernel<OUT, TS, CUT><<<grid, 256, 0, a.stream>>>(                                      \
        (const _Float16*)a.A, (const _Float16*)a.B, a.C, a.offsets, groups, rows, M, N, (int)tiles_m, \
        (int)tiles_n, MxOperand{})
#define LIBGEMM_TILE(OUT, TS)                          \
    do {                                               \
        if (M % 8 || N % 8) LIBGEMM_CUT(OUT, TS, true); \
        else LIBGEMM_CUT(OUT, TS, false);              \
    } while (0)
    const bool f32 = a.out_dtype == OUT_F32;
    if (size == 256) {
        if (f32 && lines) LIBGEMM_PP(OUT_F32, true);
        else if (f32) LIBGEMM_PP(OUT_F32, false);
        else if (lines) LIBGEMM_PP(OUT_F16, true);
        else LIBGEMM_PP(OUT_F16, false);
    } else if (size == 128) {
        if (f32) LIBGEMM_TILE(OUT_F32, 128);
        else LIBGEMM_TILE(OUT_F16, 128);
    } else {
        if (f32) LIBGEMM_TILE(OUT_F32, 64);
        else LIBGEMM_TILE(OUT_F16, 64);
    }
#undef LIBGEMM_PP
#undef LIBGEMM_TILE
#undef LIBGEMM_CUT
    return hipGetLastError();
}

}  // namespace libgemm
