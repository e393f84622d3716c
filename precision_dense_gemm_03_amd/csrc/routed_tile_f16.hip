// Grouped and adapter products on the register-staged tile kernel: FP16.
#include "routed_tile_impl.h"

namespace libgemm {

hipError_t launch_grouped_tile_f16(const GroupedArgs& a, int bm) {
    if (bm == 128)
        return a.b_kmajor ? routed::launch_grouped_tile<2, 128, 0, 0, true>(a)
                          : routed::launch_grouped_tile<2, 128, 0, 0, false>(a);
    return a.b_kmajor ? routed::launch_grouped_tile<2, 64, 0, 0, true>(a)
                      : routed::launch_grouped_tile<2, 64, 0, 0, false>(a);
}

hipError_t launch_lora_tile_f16(const LoraArgs& a, int bm) {
    return bm == 128 ? routed::launch_lora_tile<2, 128, 0, 0>(a) : routed::launch_lora_tile<2, 64, 0, 0>(a);
}

}  // namespace libgemm
