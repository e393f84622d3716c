// Grouped and adapter products on the register-staged tile kernel: FP8.
#include "routed_tile_impl.h"

namespace libgemm {

hipError_t launch_grouped_tile_fp8(const GroupedArgs& a, int bm) {
    if (bm == 128)
        return a.b_kmajor ? routed::grouped_tile_fp8<128, true>(a) : routed::grouped_tile_fp8<128, false>(a);
    return a.b_kmajor ? routed::grouped_tile_fp8<64, true>(a) : routed::grouped_tile_fp8<64, false>(a);
}

hipError_t launch_lora_tile_fp8(const LoraArgs& a, int bm) {
    return bm == 128 ? routed::lora_tile_fp8<128>(a) : routed::lora_tile_fp8<64>(a);
}

}  // namespace libgemm
