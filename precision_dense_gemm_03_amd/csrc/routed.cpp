// Which kernel runs a product whose weight depends on the row (host only, no
// HIP calls). LIBGEMM_CONFIG=<name> replaces the choice where that kernel takes
// the operands: grouped_pp_256, grouped_pp_128, grouped_ring, grouped_tile_128,
// grouped_tile_64, lora_pp_256, lora_pp_192, lora_ring, lora_tile_128,
// lora_tile_64.
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

// Time in us that a grouped kernel is expected to take; the host knows the rows
// and the number of groups, not the sizes, so it assumes half a row of tiles
// padded in each group that can have a row. A tile costs per_k ns per element
// of K (half as much again less when a compute unit runs one of two), `slots`
// run at once, and the weights stream at no more than tb TB/s. Measured on
// [rows, 2048] x [2048, 2048] in 32 groups of 2 to 256 rows and on 16384 x
// 12288 x 4096 in 16 groups.
struct Cost {
    int bm, bn;
    int64_t slots;
    double per_k, tb, fixed;
};

double estimate(const Cost& c, const GroupedArgs& a, int64_t es) {
    const double live = (double)(a.groups < a.M ? a.groups : a.M);
    double rows_t = (double)a.M / c.bm + 0.5 * live;
    if (rows_t < live) rows_t = live;
    const double tiles = rows_t * (double)ceil_div(a.N, c.bn);
    double rounds = tiles / (double)c.slots;
    if (rounds < 1.0) rounds = c.slots > kCus && tiles <= (double)kCus ? 0.6 : 1.0;
    else rounds += 0.3;   // the last round is seldom full
    const double compute = rounds * (double)a.K * c.per_k * 1e-3;
    const double stream = live * (double)a.N * (double)a.K * (double)es / (c.tb * 1e6);
    return (compute > stream ? compute : stream) + c.fixed;
}

}  // namespace

hipError_t launch_grouped(int kind, const GroupedArgs& a) {
    const bool f16 = kind == KIND_F16, bt = a.b_kmajor != 0;
    const bool mixed = a.fmt_a || a.fmt_b;
    const bool pp_ok = f16 ? grouped_pp_takes_f16(a) : grouped_pp_takes_fp8(a);
    const bool ring_ok = f16 ? grouped_ring_takes_f16(a) : grouped_ring_takes_fp8(a);
    auto pp = [&](int bm) {
        return f16 ? launch_grouped_pp_f16(a, bm) : (mixed ? launch_grouped_pp_mixed(a) : launch_grouped_pp_e4m3(a, bm));
    };
    auto ring = [&] { return f16 ? launch_grouped_ring_f16(a) : launch_grouped_ring_fp8(a); };
    auto tile = [&](int bm) { return f16 ? launch_grouped_tile_f16(a, bm) : launch_grouped_tile_fp8(a, bm); };
    const Named named;
    if (pp_ok && named("grouped_pp_256")) return pp(256);
    if (pp_ok && named("grouped_pp_128")) return pp(128);
    if (ring_ok && named("grouped_ring")) return ring();
    if (named("grouped_tile_128")) return tile(128);
    if (named("grouped_tile_64")) return tile(64);
    // The ping-pong kernel's 64-byte pieces of K-major rows stream a weight
    // that nothing shares at 3.9 TB/s (row-major 5.5), the deep ring's whole
    // lines at 5.8; row-major FP8 comes in 64-byte pieces there (2.6).
    const Cost c_pp = f16 ? Cost{256, 256, 256, 26.0, bt ? 3.9 : 5.5, 8.0} : Cost{256, 256, 256, 13.0, bt ? 3.9 : 5.5, 8.0};
    const Cost c_ring = f16 ? Cost{64, 64, 512, 10.4, bt ? 5.8 : 5.0, 4.0} : Cost{64, 64, 512, 6.3, bt ? 5.8 : 2.6, 4.0};
    const Cost c_tile = f16 ? Cost{128, 128, 512, 17.7, bt ? 4.2 : 4.6, 4.0} : Cost{128, 128, 512, 12.0, bt ? 4.2 : 2.3, 4.0};
    const int64_t es = f16 ? 2 : 1;
    const double t_pp = pp_ok ? estimate(c_pp, a, es) : 1e30;
    const double t_ring = ring_ok ? estimate(c_ring, a, es) : 1e30;
    const double t_tile = estimate(c_tile, a, es);
    // Groups of 96 to 191 rows on average take tiles of 128 rows (dgrad of 32
    // groups, 5003 x 1416 x 2048: 79 against 88 us with 256; at 64 rows on
    // average 94 against 79, at 256 134 against 115).
    if (t_pp <= t_ring && t_pp <= t_tile) return pp(a.M >= 96 * a.groups && a.M < 192 * a.groups ? 128 : 256);
    if (t_ring <= t_tile) return ring();
    return tile(a.M >= 64 * a.groups ? 128 : 64);
}

hipError_t launch_lora(int kind, const LoraArgs& call) {
    LoraArgs a = call;
    a.low_slices = lora_low_slices(a);
    const hipError_t e = launch_lora_low(a);
    if (e != hipSuccess) return e;
    const bool f16 = kind == KIND_F16, mixed = a.fmt_a || a.fmt_b;
    const bool ring_ok = f16 ? lora_ring_takes_f16(a) : lora_ring_takes_fp8(a);
    const bool pp_ok = f16 ? lora_pp_takes_f16(a) : lora_pp_takes_fp8(a);
    auto pp = [&](int bm) {
        return f16 ? launch_lora_pp_f16(a, bm) : (mixed ? launch_lora_pp_mixed(a) : launch_lora_pp_e4m3(a, bm));
    };
    auto ring = [&] { return f16 ? launch_lora_ring_f16(a) : launch_lora_ring_fp8(a); };
    auto tile = [&](int bm) { return f16 ? launch_lora_tile_f16(a, bm) : launch_lora_tile_fp8(a, bm); };
    const Named named;
    if (pp_ok && named("lora_pp_256")) return pp(256);
    if (pp_ok && named("lora_pp_192")) return pp(192);
    if (ring_ok && named("lora_ring")) return ring();
    if (named("lora_tile_128")) return tile(128);
    if (named("lora_tile_64")) return tile(64);
    // The plain product's rules (selector.cpp): the deep ring up to 256 rows;
    // 256-column tiles from 3/4 of the compute units, 192 rows high when that
    // leaves each unit fewer rows; 128 or 64 square below.
    if (a.M <= 256 && ring_ok) return ring();
    const int64_t tn = ceil_div(a.N, 256), tiles256 = ceil_div(a.M, 256) * tn, tiles192 = ceil_div(a.M, 192) * tn;
    const double useful = (double)a.M * (double)a.N;
    if (pp_ok && tiles256 <= 0x7FFFFFFF && tiles256 >= kCus * 3 / 4 && useful >= 0.75 * 65536.0 * (double)tiles256)
        return pp(ceil_div(tiles192, kCus) * 192 < ceil_div(tiles256, kCus) * 256 ? 192 : 256);
    return tile(ceil_div(a.M, 128) * ceil_div(a.N, 128) >= kCus ? 128 : 64);
}

}  // namespace libgemm
