// Estimated times of the kernels that run one product for all rows (host only).
#pragma once

#include <cstdint>

namespace libgemm {

constexpr int64_t kCus = 256;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// One weight for all rows, with adapters (rank) or without (rank 0: what they cost
// is left out): the sizes are known. 256-column tiles come in whole rounds; the
// low-rank term costs `term` us a round and 32 of rank; the deep ring's rounds
// are the bytes of its chosen tile (ring_cost, 64 x 64: 128) and its term us
// per million of rows x columns x rank.
struct LoraCost {
    int bm, bn;
    double per_k, least, more, term, fixed;
};

enum { L_PP_256, L_PP_192, L_RING, L_TILE_128, L_TILE_64, N_LORA };

constexpr LoraCost kLora[2][N_LORA] = {{{256, 256, 30.3, 0, 0, 1.4, 18.0},
                                        {192, 256, 21.1, 0, 0, 4.0, 18.0},
                                        {0, 0, 8.3, 0.32, 0, 0.40, 9.9},
                                        {128, 128, 10.8, 0.21, 1.16, 2.1, 18.0},
                                        {64, 64, 4.9, 1.49, 0.09, 0.64, 13.0}},
                                       {{256, 256, 21.8, 0, 0, 0.15, 18.0},
                                        {192, 256, 16.0, 0, 0, 4.0, 18.0},
                                        {0, 0, 5.1, 0.20, 0, 0.45, 12.9},
                                        {128, 128, 8.6, 0.96, 0.01, 4.0, 18.0},
                                        {64, 64, 3.1, 1.46, 0.48, 0.23, 12.9}}};

inline double estimate(int which, const LoraCost& c, int64_t M, int64_t N, int64_t K, int64_t rank, int64_t ring_cost) {
    const double k = (double)K * 1e-3;
    if (which == L_RING) {
        double rounds = (double)ring_cost / 128.0;
        if (rounds < c.least) rounds = c.least;
        return rounds * k * c.per_k + c.fixed + (double)M * (double)N * (double)rank * c.term * 1e-6;
    }
    const int64_t tiles = ceil_div(M, c.bm) * ceil_div(N, c.bn);
    double rounds;
    if (c.bn == 256) {
        rounds = (double)ceil_div(tiles, kCus);
    } else {
        rounds = (double)tiles / (double)kCus + c.more;
        if (rounds < c.least) rounds = c.least;
    }
    const double share = tiles > kCus ? (double)tiles / (double)kCus : 1.0;
    return rounds * k * c.per_k + c.fixed + share * (double)ceil_div(rank, 32) * c.term;
}

}  // namespace libgemm
