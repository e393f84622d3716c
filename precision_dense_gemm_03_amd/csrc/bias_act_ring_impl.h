// Products with bias, activation and residual on the deep-ring kernel
// (gemm_ring_impl.h), with the tiles and the K tiles per barrier that the adapters'
// products measured fastest. Few rows are bound by the weight's stream: 4 x 12288 x
// 4096 FP16, K-major, with bias and SILU 18.8 us, 5.4 TB/s.
#pragma once

#include "bias_act_extra.h"
#include "gemm_ring_impl.h"

namespace libgemm {
namespace bias_act {

template <int BM, int BN>
struct RingShape {
    static constexpr int P = BM * BN <= 512 ? 4 : 2;
    static constexpr int FIT = 128 * 1024 / ((BM + BN) * 128), S = (FIT < 12 ? FIT : 12) / P * P;
};

template <int ES, int BM, int BN, int FA, int FB, bool BT>
__global__ __launch_bounds__(256) void bias_act_ring_kernel(const uint8_t* __restrict__ A,
                                                            const uint8_t* __restrict__ B, int M, int N, int K,
                                                            int tiles_m, int tiles_n, BiasActExtra<> ext) {
    constexpr int S = RingShape<BM, BN>::S, P = RingShape<BM, BN>::P;
    using T = ring::Ring<ES, BM, BN, BT, S>;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[T::S * T::STAGE];
    __shared__ v4f red[T::RED_SLOTS];
    if (past_last_block((int64_t)tiles_m * tiles_n)) return;
    int tm, tn;
    tile_coords((int)wide_block(), tiles_m, tiles_n, tm, tn);
    ring::ring_body<ES, BM, BN, OUT_F32, FA, FB, BT, S, true, BiasActExtra<>, P>(
        A, B, nullptr, M, N, K, nullptr, nullptr, nullptr, tm * BM, tn * BN, 0, 0, ring, red, ext);
}

template <int ES, int FA, int FB, bool BT, int BM, int BN>
hipError_t launch_ring(const BiasActArgs& a) {
    const int64_t tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN;
    if (tiles_m * tiles_n > kMostWorkgroups) return hipErrorInvalidValue;
    bias_act_ring_kernel<ES, BM, BN, FA, FB, BT><<<wide_grid(tiles_m * tiles_n), 256, 0, a.stream>>>(
        reinterpret_cast<const uint8_t*>(a.A), reinterpret_cast<const uint8_t*>(a.B), (int)a.M, (int)a.N, (int)a.K,
        (int)tiles_m, (int)tiles_n, bias_act_extra(a));
    return hipGetLastError();
}

// shape: of kLoraRingShapes.
template <int ES, int FA, int FB, bool BT>
hipError_t launch_ring_shape(const BiasActArgs& a, int shape) {
    switch (shape) {
        case 0: return launch_ring<ES, FA, FB, BT, 16, 16>(a);
        case 1: return launch_ring<ES, FA, FB, BT, 16, 32>(a);
        case 2: return launch_ring<ES, FA, FB, BT, 16, 64>(a);
        case 3: return launch_ring<ES, FA, FB, BT, 32, 32>(a);
        case 4: return launch_ring<ES, FA, FB, BT, 32, 64>(a);
        default: return launch_ring<ES, FA, FB, BT, 64, 64>(a);
    }
}

}  // namespace bias_act
}  // namespace libgemm
