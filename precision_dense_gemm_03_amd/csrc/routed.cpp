// Which kernel runs a product whose weight depends on the row (host only).
#include "kernels.h"

namespace libgemm {

hipError_t launch_grouped(int kind, const GroupedArgs& a) {
    const int bm = a.M >= 128 * a.groups ? 128 : 64;
    return kind == KIND_F16 ? launch_grouped_tile_f16(a, bm) : launch_grouped_tile_fp8(a, bm);
}

hipError_t launch_lora(int kind, const LoraArgs& a) {
    const hipError_t e = launch_lora_low(a);
    if (e != hipSuccess) return e;
    const int bm = ((a.M + 127) / 128) * ((a.N + 127) / 128) >= 256 ? 128 : 64;
    return kind == KIND_F16 ? launch_lora_tile_f16(a, bm) : launch_lora_tile_fp8(a, bm);
}

}  // namespace libgemm
