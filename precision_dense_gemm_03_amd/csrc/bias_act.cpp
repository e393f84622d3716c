// Which kernel runs a product with bias, activation and residual (host only, no
// HIP calls). LIBGEMM_CONFIG=<name> replaces the choice where that kernel takes the
// operands: bias_act_pp_256, bias_act_pp_192, bias_act_ring, bias_act_tile_128,
// bias_act_tile_64, bias_act_gemv.
#include <cstdlib>
#include <cstring>

#include "kernels.h"

namespace libgemm {

namespace {

constexpr int64_t kCus = 256;
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

enum { PP_256, PP_192, RING, TILE_128, TILE_64, GEMV };
constexpr const char* kNames[] = {"bias_act_pp_256", "bias_act_pp_192", "bias_act_ring",
                                  "bias_act_tile_128", "bias_act_tile_64", "bias_act_gemv"};

// Estimated us, fits to measured times of 2600 shapes (1 to 16384 rows, 128 to 12288
// columns, K from 128 to 8192, odd sizes among them, weights from beyond the caches):
// choosing by them costs 1.0 to 1.2 % over the fastest of each shape, by the adapters'
// constants (routed.cpp) 2.4 %. Rounds of tiles over compute units (the ping-pong
// kernel's whole, one workgroup per unit; the others' with `more` for the uneven end
// and no less than `least`; the deep ring's by its tile's bytes, 64 x 64: 1) take per_k
// ns each for an element of K and `epi` us, the ping-pong and 64-row kernels' more by
// `odd` where rows of C are no multiple of 8 values; operands stream at tb TB/s.
struct Cost {
    int bm, bn;
    double per_k, least, more, epi, tb, fixed, odd;
};
constexpr double kFree = 1e3;

// [FP16, FP8][row-major, K-major]
constexpr Cost kCosts[2][2][5] = {
    {{{256, 256, 15.76, 0, 0, 14.47, kFree, 0, 0.95},
      {192, 256, 13.86, 0, 0, 12.91, kFree, 0, 2.87},
      {0, 0, 5.82, 0.4, 0, 3.1, kFree, 4.36, 0},
      {128, 128, 12.33, 1.01, 0.45, 4.85, kFree, 5.05, 0},
      {64, 64, 3.52, 1.76, 1, 1.02, 2.38, 3.49, 0.28}},
     {{256, 256, 16.98, 0, 0, 12.44, 0.78, 0, 0.38},
      {192, 256, 15.29, 0, 0, 11.25, 0.87, 0, 0.33},
      {0, 0, 5.35, 0.25, 0, 2.56, 11.88, 4.82, 1},
      {128, 128, 12.12, 1, 0.3, 4.79, kFree, 5.16, 0},
      {64, 64, 3.55, 1.44, 0.79, 0.95, 2.08, 3.87, 0}}},
    {{{256, 256, 9.1, 0, 0, 15, kFree, 0, 1.03},
      {192, 256, 7.87, 0, 0, 12.9, kFree, 0, 0.06},
      {0, 0, 3.63, 0.53, 0, 3.37, kFree, 5.2, 0},
      {128, 128, 9.88, 0.69, 0, 15.18, kFree, 3.97, 0},
      {64, 64, 2.63, 1, 0.28, 1.21, kFree, 5.98, 0.31}},
     {{256, 256, 9.21, 0, 0, 13.25, 0.71, 0, 0.57},
      {192, 256, 8.59, 0, 0, 11.68, kFree, 0, 0.56},
      {0, 0, 2.69, 0.2, 0, 2.76, 5.5, 6.36, 1},
      {128, 128, 6.5, 0.93, 0.24, 7.38, kFree, 7.22, 0.07},
      {64, 64, 2.07, 1, 0.13, 1.25, 2.31, 6.18, 0}}}};

double estimate(const Cost& c, const BiasActArgs& a, int64_t es, int64_t ring_cost) {
    double rounds;
    if (c.bn == 256) {
        rounds = (double)ceil_div(ceil_div(a.M, c.bm) * ceil_div(a.N, c.bn), kCus);
    } else {
        rounds = c.bm == 0 ? (double)ring_cost / 128.0
                           : (double)(ceil_div(a.M, c.bm) * ceil_div(a.N, c.bn)) / (double)kCus + c.more;
        if (rounds < c.least) rounds = c.least;
    }
    const double compute = rounds * ((double)a.K * c.per_k * 1e-3 + c.epi * (a.N % 8 ? 1.0 + c.odd : 1.0));
    const double stream = ((double)a.N + (double)a.M) * (double)a.K * (double)es / (c.tb * 1e6);
    return (compute > stream ? compute : stream) + c.fixed;
}

// 8-bit values of z need waves that hold 32 columns: the deep ring's tiles from 32 x 64 on.
constexpr int kFirstMxShape = 4;

bool mx(const BiasActArgs& a) { return a.Z && a.z_dtype >= 2 /* 8-bit values */; }

// The deep ring's tile: the fewest bytes a compute unit streams (lora_ring_shape).
int ring_shape(const BiasActArgs& a, int64_t* cost) {
    if (!mx(a)) return lora_ring_shape(a.M, a.N, cost);
    int pick = -1;
    for (int i = kFirstMxShape; i < 6; ++i) {
        const int* c = kLoraRingShapes[i];
        const int64_t bytes = ceil_div(ceil_div(a.M, c[0]) * ceil_div(a.N, c[1]), kCus) * (c[0] + c[1]);
        if (pick < 0 || bytes <= *cost) {
            pick = i;
            *cost = bytes;
        }
    }
    return pick;
}

int choose(int kind, const BiasActArgs& a) {
    const bool f16 = kind == KIND_F16, mixed = a.fmt_a || a.fmt_b;   // (one height on the ping-pong kernel: 192 rows)
    if (a.K <= 0) return TILE_64;
    const bool pp_ok = f16 ? bias_act_pp_takes_f16(a) : bias_act_pp_takes_fp8(a);
    const bool ring_ok = bias_act_ring_takes(kind, a);
    // One FP16 row meets a K-major weight in the decode kernel: 0.90 of the time of the
    // others over 33 shapes; one to four FP8 rows there 1.01 to 1.12. (The launch holds one
    // workgroup per four columns.)
    const bool gemv_ok = f16 && a.b_kmajor && a.M <= 1 && !mx(a) && a.N < (1 << 25);
    if (const char* env = std::getenv("LIBGEMM_CONFIG")) {
        for (int i = 0; i <= GEMV; ++i) {
            if (std::strcmp(env, kNames[i]) != 0) continue;
            if (i == PP_256 && pp_ok) return mixed ? PP_192 : PP_256;
            if ((i == PP_192 && pp_ok) || (i == RING && ring_ok) || (i == GEMV && gemv_ok) || i == TILE_128 ||
                i == TILE_64)
                return i;
        }
    }
    if (gemv_ok) return GEMV;
    int64_t cost = 0;
    ring_shape(a, &cost);
    int best = -1;
    double least = 0.0;
    for (int i = 0; i < GEMV; ++i) {
        if ((i == PP_256 || i == PP_192) && !pp_ok) continue;
        if (i == PP_256 && mixed) continue;
        if (i == RING && !ring_ok) continue;
        const double t = estimate(kCosts[f16 ? 0 : 1][a.b_kmajor ? 1 : 0][i], a, f16 ? 2 : 1, cost);
        if (best < 0 || t < least) {
            best = i;
            least = t;
        }
    }
    return best;
}

}  // namespace

const char* bias_act_kernel_name(int kind, const BiasActArgs& a) { return kNames[choose(kind, a)]; }

hipError_t launch_bias_act(int kind, const BiasActArgs& a) {
    const bool f16 = kind == KIND_F16, mixed = a.fmt_a || a.fmt_b;
    auto pp = [&](int bm) {
        return f16 ? launch_bias_act_pp_f16(a, bm) : (mixed ? launch_bias_act_pp_mixed(a) : launch_bias_act_pp_e4m3(a, bm));
    };
    auto tile = [&](int bm) { return f16 ? launch_bias_act_tile_f16(a, bm) : launch_bias_act_tile_fp8(a, bm); };
    switch (choose(kind, a)) {
        case PP_256: return pp(256);
        case PP_192: return pp(192);
        case RING: {
            int64_t cost = 0;
            const int shape = ring_shape(a, &cost);
            return f16 ? launch_bias_act_ring_f16(a, shape) : launch_bias_act_ring_fp8(a, shape);
        }
        case TILE_128: return tile(128);
        case GEMV: return launch_bias_act_gemv_f16(a);
        default: return tile(64);
    }
}

}  // namespace libgemm
