// Which kernel runs a product whose weight depends on the row (host only, no
// HIP calls). LIBGEMM_CONFIG=<name> replaces the choice where that kernel takes
// the operands: grouped_pp_256, grouped_pp_192, grouped_pp_128, grouped_ring,
// grouped_tile_128, grouped_tile_64, lora_pp_256, lora_pp_192, lora_ring,
// lora_tile_128, lora_tile_64.
#include <cstdlib>
#include <cstring>

#include "kernels.h"

namespace libgemm {

namespace {

constexpr int64_t kCus = 256;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether the environment names this kernel (looked up once per call).
struct Named {
    const char* env = std::getenv("LIBGEMM_CONFIG");
    bool operator()(const char* name) const { return env && std::strcmp(env, name) == 0; }
};

// Estimated times in us. The constants are fits to measured times of every
// kernel on 60 to 110 shapes per table, from 1 to 16384 rows, with weights that
// come from beyond the caches; choosing by them costs 1 to 3 % over choosing
// the fastest of each shape after the fact (fixed bounds on rows per group
// cost 5 to 12 %). Terms that are the same for every kernel are left out.
//
// Grouped: the host knows the rows and the number of groups, not the sizes,
// and assumes half a row of tiles padded in each group that can have a row.
// Tiles over compute units, and `more` for the uneven end, but no less than
// `least` (one tile alone), take per_k ns each per element of K; the weights
// stream at no more than tb TB/s.
struct Cost {
    int bm, bn;
    double per_k, least, more, tb, fixed;
};

double estimate(const Cost& c, const GroupedArgs& a, int64_t es) {
    const double live = (double)(a.groups < a.M ? a.groups : a.M);
    double rows_t = (double)a.M / c.bm + 0.5 * live;
    if (rows_t < live) rows_t = live;
    double rounds = rows_t * (double)ceil_div(a.N, c.bn) / (double)kCus + c.more;
    if (rounds < c.least) rounds = c.least;
    const double compute = rounds * (double)a.K * c.per_k * 1e-3;
    const double stream = live * (double)a.N * (double)a.K * (double)es / (c.tb * 1e6);
    return (compute > stream ? compute : stream) + c.fixed;
}

enum { PP_256, PP_128, RING, TILE_128, TILE_64, N_GROUPED };

// [FP16, FP8][row-major, K-major]. K-major weights that nothing shares stream
// fastest in the deep ring's whole lines; row-major FP8 comes in 64-byte pieces.
constexpr Cost kGrouped[2][2][N_GROUPED] = {
    {{{256, 256, 32.7, 0.21, 0.35, 3.4, 9.0},
      {128, 256, 28.0, 0.43, 0.04, 3.7, 9.0},
      {64, 64, 7.9, 0.48, 0.08, 5.9, 5.4},
      {128, 128, 20.3, 0.60, 0.03, 5.1, 7.7},
      {64, 64, 5.9, 1.15, 0.64, 4.7, 4.9}},
     {{256, 256, 14.1, 0.30, 1.04, 3.9, 9.0},
      {128, 256, 27.6, 0.62, 0.08, 3.6, 7.3},
      {64, 64, 5.2, 0.62, 0.02, 6.7, 6.0},
      {128, 128, 11.2, 1.10, 0.03, 4.3, 6.3},
      {64, 64, 4.6, 1.46, 0.01, 4.7, 4.4}}},
    {{{256, 256, 12.3, 0.24, 0.57, 5.2, 9.0},
      {128, 256, 20.1, 0.19, 0.24, 7.5, 9.0},
      {64, 64, 5.6, 0.31, 0.02, 5.4, 9.0},
      {128, 128, 9.4, 0.24, 0.53, 4.3, 9.0},
      {64, 64, 3.9, 0.14, 0.35, 6.6, 6.9}},
     {{256, 256, 11.5, 0.14, 0.96, 5.5, 9.0},
      {128, 256, 14.1, 0.13, 0.53, 6.1, 9.0},
      {64, 64, 2.7, 0.28, 0.09, 7.5, 9.0},
      {128, 128, 8.6, 0.41, 0.33, 5.8, 9.0},
      {64, 64, 2.4, 0.16, 0.78, 4.8, 6.9}}}};

// Whether 192 rows a tile beat 256: a round of them takes 0.91 of the time, and
// the end of a launch costs between the part of a round it fills and a whole
// one. 8192 rows in 8 groups, 4096 x 4096 FP16: 285 against 304 us (2.9 rounds
// against 2.25); 3000 rows in 4 groups: 154 against 104 (1.1 against 0.86).
bool shorter_tiles(const GroupedArgs& a) {
    auto rounds = [&](double bm) {
        const double x = ((double)a.M / bm + 0.5 * (double)a.groups) * (double)ceil_div(a.N, 256) / (double)kCus;
        const double whole = (double)(int64_t)x + (x > (double)(int64_t)x ? 1.0 : 0.0);
        return x < 1.0 ? 1.0 : 0.35 * x + 0.65 * whole;
    };
    return 0.91 * rounds(192.0) < rounds(256.0);
}

// Adapters: the sizes are known. 256-column tiles come in whole rounds; the
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

double estimate(int which, const LoraCost& c, const LoraArgs& a, int64_t ring_cost) {
    const double k = (double)a.K * 1e-3;
    if (which == L_RING) {
        double rounds = (double)ring_cost / 128.0;
        if (rounds < c.least) rounds = c.least;
        return rounds * k * c.per_k + c.fixed + (double)a.M * (double)a.N * (double)a.rank * c.term * 1e-6;
    }
    const int64_t tiles = ceil_div(a.M, c.bm) * ceil_div(a.N, c.bn);
    double rounds;
    if (c.bn == 256) {
        rounds = (double)ceil_div(tiles, kCus);
    } else {
        rounds = (double)tiles / (double)kCus + c.more;
        if (rounds < c.least) rounds = c.least;
    }
    const double share = tiles > kCus ? (double)tiles / (double)kCus : 1.0;
    return rounds * k * c.per_k + c.fixed + share * (double)ceil_div(a.rank, 32) * c.term;
}

// The kernels by name, in the order of the enums.
enum GroupedKernel { G_PP_256, G_PP_192, G_PP_128, G_RING, G_TILE_128, G_TILE_64 };
constexpr const char* kGroupedNames[] = {"grouped_pp_256", "grouped_pp_192", "grouped_pp_128",
                                         "grouped_ring", "grouped_tile_128", "grouped_tile_64"};
constexpr const char* kLoraNames[N_LORA] = {"lora_pp_256", "lora_pp_192", "lora_ring", "lora_tile_128", "lora_tile_64"};

GroupedKernel choose_grouped(int kind, const GroupedArgs& a) {
    const bool f16 = kind == KIND_F16, bt = a.b_kmajor != 0;
    const bool mixed = a.fmt_a || a.fmt_b;   // (one height on the ping-pong kernel: 192 rows)
    const bool pp_ok = f16 ? grouped_pp_takes_f16(a) : grouped_pp_takes_fp8(a);
    const bool ring_ok = f16 ? grouped_ring_takes_f16(a) : grouped_ring_takes_fp8(a);
    const Named named;
    if (pp_ok && named("grouped_pp_256")) return mixed ? G_PP_192 : G_PP_256;
    if (pp_ok && named("grouped_pp_192")) return G_PP_192;
    if (pp_ok && named("grouped_pp_128")) return mixed ? G_PP_192 : G_PP_128;
    if (ring_ok && named("grouped_ring")) return G_RING;
    if (named("grouped_tile_128")) return G_TILE_128;
    if (named("grouped_tile_64")) return G_TILE_64;
    int best = -1;
    double least = 0.0;
    for (int i = 0; i < N_GROUPED; ++i) {
        if ((i == PP_256 || i == PP_128) && (!pp_ok || (i == PP_128 && mixed))) continue;
        if (i == RING && !ring_ok) continue;
        const double t = estimate(kGrouped[f16 ? 0 : 1][bt ? 1 : 0][i], a, f16 ? 2 : 1);
        if (best < 0 || t < least) {
            best = i;
            least = t;
        }
    }
    switch (best) {
        case PP_256: return mixed || shorter_tiles(a) ? G_PP_192 : G_PP_256;
        case PP_128: return G_PP_128;
        case RING: return G_RING;
        case TILE_128: return G_TILE_128;
        default: return G_TILE_64;
    }
}

int choose_lora(int kind, const LoraArgs& a) {
    const bool f16 = kind == KIND_F16, mixed = a.fmt_a || a.fmt_b;   // (as above)
    const bool ring_ok = f16 ? lora_ring_takes_f16(a) : lora_ring_takes_fp8(a);
    const bool pp_ok = f16 ? lora_pp_takes_f16(a) : lora_pp_takes_fp8(a);
    const Named named;
    if (pp_ok && named("lora_pp_256")) return mixed ? L_PP_192 : L_PP_256;
    if (pp_ok && named("lora_pp_192")) return L_PP_192;
    if (ring_ok && named("lora_ring")) return L_RING;
    if (named("lora_tile_128")) return L_TILE_128;
    if (named("lora_tile_64")) return L_TILE_64;
    int64_t cost = 0;
    lora_ring_shape(a.M, a.N, &cost);
    int best = -1;
    double least = 0.0;
    for (int i = 0; i < N_LORA; ++i) {
        if ((i == L_PP_256 || i == L_PP_192) && !pp_ok) continue;
        if (i == L_PP_256 && mixed) continue;
        if (i == L_RING && !ring_ok) continue;
        const double t = estimate(i, kLora[f16 ? 0 : 1][i], a, cost);
        if (best < 0 || t < least) {
            best = i;
            least = t;
        }
    }
    return best;
}

}  // namespace

const char* grouped_kernel_name(int kind, const GroupedArgs& a) { return kGroupedNames[choose_grouped(kind, a)]; }
const char* lora_kernel_name(int kind, const LoraArgs& a) { return kLoraNames[choose_lora(kind, a)]; }

hipError_t launch_grouped(int kind, const GroupedArgs& a) {
    const bool f16 = kind == KIND_F16, mixed = a.fmt_a || a.fmt_b;
    auto pp = [&](int bm) {
        return f16 ? launch_grouped_pp_f16(a, bm) : (mixed ? launch_grouped_pp_mixed(a) : launch_grouped_pp_e4m3(a, bm));
    };
    auto tile = [&](int bm) { return f16 ? launch_grouped_tile_f16(a, bm) : launch_grouped_tile_fp8(a, bm); };
    switch (choose_grouped(kind, a)) {
        case G_PP_256: return pp(256);
        case G_PP_192: return pp(192);
        case G_PP_128: return pp(128);
        case G_RING: return f16 ? launch_grouped_ring_f16(a) : launch_grouped_ring_fp8(a);
        case G_TILE_128: return tile(128);
        default: return tile(64);
    }
}

hipError_t launch_lora(int kind, const LoraArgs& call) {
    LoraArgs a = call;
    a.low_slices = lora_low_slices(a);
    const hipError_t e = launch_lora_low(a);
    if (e != hipSuccess) return e;
    const bool f16 = kind == KIND_F16, mixed = a.fmt_a || a.fmt_b;
    auto pp = [&](int bm) {
        return f16 ? launch_lora_pp_f16(a, bm) : (mixed ? launch_lora_pp_mixed(a) : launch_lora_pp_e4m3(a, bm));
    };
    auto tile = [&](int bm) { return f16 ? launch_lora_tile_f16(a, bm) : launch_lora_tile_fp8(a, bm); };
    switch (choose_lora(kind, a)) {
        case L_PP_256: return pp(256);
        case L_PP_192: return pp(192);
        case L_RING: return f16 ? launch_lora_ring_f16(a) : launch_lora_ring_fp8(a);
        case L_TILE_128: return tile(128);
        default: return tile(64);
    }
}

}  // namespace libgemm
