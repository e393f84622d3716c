// Products with bias, activation and residual on the register-staged tile kernel
// (gemm_tile_impl.h), which takes operands of any size and alignment. Bound by its
// tile loop: 3343 x 6592 x 4005 FP16, K-major, 323 us, 0.57 PFLOP/s; 7895 x 3872 x
// 5621 FP8 373 us, 0.94.
#include "bias_act_extra.h"
#include "gemm_tile_impl.h"
#include "wide_grid.h"

namespace libgemm {

namespace {

template <int ES, int BM, int FA, int FB, bool BT>
__global__ __launch_bounds__(256) void bias_act_tile_kernel(const uint8_t* __restrict__ A,
                                                            const uint8_t* __restrict__ B, int M, int N, int K,
                                                            int tiles_m, int tiles_n, BiasActExtra<> ext) {
    if (past_last_block((int64_t)tiles_m * tiles_n)) return;
    int tm, tn;
    tile_coords((int)wide_block(), tiles_m, tiles_n, tm, tn);
    tile::tile_body<ES, OUT_F32, BM, BM, 128 / ES, 2, 2, FA, FB, BT, ES, true, BiasActExtra<>>(
        A, B, nullptr, M, N, K, nullptr, nullptr, nullptr, tm * BM, tn * BM, 1, 0, K, 0, ext);
}

template <int ES, int BM, int FA, int FB, bool BT>
hipError_t launch(const BiasActArgs& a) {
    const int64_t tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BM - 1) / BM;
    if (tiles_m * tiles_n > kMostWorkgroups) return hipErrorInvalidValue;
    bias_act_tile_kernel<ES, BM, FA, FB, BT><<<wide_grid(tiles_m * tiles_n), 256, 0, a.stream>>>(
        reinterpret_cast<const uint8_t*>(a.A), reinterpret_cast<const uint8_t*>(a.B), (int)a.M, (int)a.N, (int)a.K,
        (int)tiles_m, (int)tiles_n, bias_act_extra(a));
    return hipGetLastError();
}

template <int BM, bool BT>
hipError_t launch_fp8(const BiasActArgs& a) {
    switch (a.fmt_a * 2 + a.fmt_b) {
        case 0: return launch<1, BM, 0, 0, BT>(a);
        case 1: return launch<1, BM, 0, 1, BT>(a);
        case 2: return launch<1, BM, 1, 0, BT>(a);
        default: return launch<1, BM, 1, 1, BT>(a);
    }
}

}  // namespace

hipError_t launch_bias_act_tile_f16(const BiasActArgs& a, int bm) {
    if (bm == 128) return a.b_kmajor ? launch<2, 128, 0, 0, true>(a) : launch<2, 128, 0, 0, false>(a);
    return a.b_kmajor ? launch<2, 64, 0, 0, true>(a) : launch<2, 64, 0, 0, false>(a);
}

hipError_t launch_bias_act_tile_fp8(const BiasActArgs& a, int bm) {
    if (bm == 128) return a.b_kmajor ? launch_fp8<128, true>(a) : launch_fp8<128, false>(a);
    return a.b_kmajor ? launch_fp8<64, true>(a) : launch_fp8<64, false>(a);
}

}  // namespace libgemm
