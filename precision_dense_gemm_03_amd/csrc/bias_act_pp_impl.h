// Products with bias, activation and residual on the ping-pong tile kernel
// (gemm_pp_impl.h), whose epilogue they replace (bias_act_extra.h). Bound by the tile
// loop; one workgroup fills a CU, so the epilogue is not hidden. On one machine 16384 x
// 12288 x 4096 FP8, per channel: 652 us without, 697 with bias and GELU_TANH, 757 to 760
// with an FP16 residual too (plain product 637; 756 to 799 over five machines); 4096^3
// FP16 with GELU and z in 8 bits 122.5 (plain 112; 122 to 130).
#pragma once

#include "bias_act_extra.h"
#include "gemm_pp_impl.h"

namespace libgemm {
namespace bias_act {

template <int ES, int FA, int FB, bool BT, int BM, bool LINES, int HOW>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void bias_act_pp_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tiles_m, int tiles_n,
    BiasActExtra<LINES, HOW> ext) {
    using T = pp::Pp<ES, BM>;
    LIBGEMM_PP_LDS(T);
    if (past_last_block((int64_t)tiles_m * tiles_n)) return;
    int tm, tn;
    tile_coords((int)wide_block(), tiles_m, tiles_n, tm, tn);
    pp::pp_body<ES, OUT_F32, FA, FB, BT, false, BM, true, BiasActExtra<LINES, HOW>>(
        A, B, nullptr, M, N, K, nullptr, nullptr, nullptr, tm * BM, tn * 256, 0, 0, lds, ext);
}

// Rows of whole 128-byte lines in every FP16 and FP32 matrix of the epilogue.
inline bool whole_lines(const BiasActArgs& a) {
    auto line = [](const void* p) { return ((uintptr_t)p & 127) == 0; };
    return a.N % 64 == 0 && line(a.C) && line(a.residual) && line(a.Z);
}

template <int ES, int FA, int FB, bool BT, int BM>
hipError_t launch_pp(const BiasActArgs& a) {
    const int64_t tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + 255) / 256;
    if (tiles_m * tiles_n > kMostWorkgroups) return hipErrorInvalidValue;
    const uint8_t* A = reinterpret_cast<const uint8_t*>(a.A);
    const uint8_t* B = reinterpret_cast<const uint8_t*>(a.B);
#define LIBGEMM_GO(LINES, HOW)                                                                              \
    bias_act_pp_kernel<ES, FA, FB, BT, BM, LINES, HOW><<<wide_grid(tiles_m * tiles_n), 512, 0, a.stream>>>( \
        A, B, (int)a.M, (int)a.N, (int)a.K, (int)tiles_m, (int)tiles_n, bias_act_extra<LINES, HOW>(a))
    const bool fine = a.out_dtype == OUT_F32 && a.act >= ACT_GELU;   // (none and RELU have one form)
    const bool lines = whole_lines(a);
    if (fine && lines) LIBGEMM_GO(true, FINE);
    else if (fine) LIBGEMM_GO(false, FINE);
    else if (lines) LIBGEMM_GO(true, COARSE);
    else LIBGEMM_GO(false, COARSE);
#undef LIBGEMM_GO
    return hipGetLastError();
}

template <int ES>
bool pp_takes(const BiasActArgs& a) {
    return a.b_kmajor ? pp::pp_fits<ES, true, 256>(a) : pp::pp_fits<ES, false, 256>(a);
}

}  // namespace bias_act
}  // namespace libgemm
