// Which kernel runs a product with bias, activation and residual (host only, no
// HIP calls). LIBGEMM_CONFIG=<name> replaces the choice where that kernel takes the
// operands: bias_act_pp_256, bias_act_pp_192, bias_act_ring, bias_act_tile_128,
// bias_act_tile_64, bias_act_gemv.
#include <cstdlib>
#include <cstring>

#include "kernels.h"
#include "product_cost.h"

namespace libgemm {

namespace {

enum { GEMV = N_LORA };   // after the kernels of product_cost.h
constexpr const char* kNames[] = {"bias_act_pp_256", "bias_act_pp_192", "bias_act_ring",
                                  "bias_act_tile_128", "bias_act_tile_64", "bias_act_gemv"};

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
    if (a.K <= 0) return L_TILE_64;
    const bool pp_ok = f16 ? bias_act_pp_takes_f16(a) : bias_act_pp_takes_fp8(a);
    const bool ring_ok = bias_act_ring_takes(kind, a);
    // (the plain products' bounds; the launch holds one workgroup per four columns)
    const bool gemv_ok = a.b_kmajor && a.M <= (f16 ? kBiasActGemvF16 : kBiasActGemvFp8) && !mx(a) && a.N < (1 << 25);
    if (const char* env = std::getenv("LIBGEMM_CONFIG")) {
        for (int i = 0; i <= GEMV; ++i) {
            if (std::strcmp(env, kNames[i]) != 0) continue;
            if (i == L_PP_256 && pp_ok) return mixed ? L_PP_192 : L_PP_256;
            if ((i == L_PP_192 && pp_ok) || (i == L_RING && ring_ok) || (i == GEMV && gemv_ok) || i == L_TILE_128 ||
                i == L_TILE_64)
                return i;
        }
    }
    if (gemv_ok) return GEMV;
    int64_t cost = 0;
    ring_shape(a, &cost);
    int best = -1;
    double least = 0.0;
    for (int i = 0; i < N_LORA; ++i) {
        if ((i == L_PP_256 || i == L_PP_192) && !pp_ok) continue;
        if (i == L_PP_256 && mixed) continue;
        if (i == L_RING && !ring_ok) continue;
        const double t = estimate(i, kLora[f16 ? 0 : 1][i], a.M, a.N, a.K, 0, cost);
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
        case L_PP_256: return pp(256);
        case L_PP_192: return pp(192);
        case L_RING: {
            int64_t cost = 0;
            const int shape = ring_shape(a, &cost);
            return f16 ? launch_bias_act_ring_f16(a, shape) : launch_bias_act_ring_fp8(a, shape);
        }
        case L_TILE_128: return tile(128);
        case GEMV: return f16 ? launch_bias_act_gemv_f16(a) : launch_bias_act_gemv_fp8(a);
        default: return tile(64);
    }
}

}  // namespace libgemm
