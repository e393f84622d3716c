// Grouped and adapter products on the ping-pong tile kernel: FP16.
#include "routed_pp_impl.h"

namespace libgemm {

bool grouped_pp_takes_f16(const GroupedArgs& a) { return routed::grouped_pp_fits<2>(a); }

hipError_t launch_grouped_pp_f16(const GroupedArgs& a, int bm) {
    switch (bm) {
        case 256: return a.b_kmajor ? routed::launch_grouped_pp<2, 0, 0, true, 256>(a)
                                    : routed::launch_grouped_pp<2, 0, 0, false, 256>(a);
        case 192: return a.b_kmajor ? routed::launch_grouped_pp<2, 0, 0, true, 192>(a)
                                    : routed::launch_grouped_pp<2, 0, 0, false, 192>(a);
        default: return a.b_kmajor ? routed::launch_grouped_pp<2, 0, 0, true, 128>(a)
                                   : routed::launch_grouped_pp<2, 0, 0, false, 128>(a);
    }
}

bool lora_pp_takes_f16(const LoraArgs& a) { return pp::pp_fits<2, true, 256>(a); }

hipError_t launch_lora_pp_f16(const LoraArgs& a, int bm) {
    return bm == 256 ? routed::launch_lora_pp<2, 0, 0, 256>(a) : routed::launch_lora_pp<2, 0, 0, 192>(a);
}

}  // namespace libgemm
