// Grouped and adapter products on the deep-ring kernel: FP8.
#include "routed_ring_impl.h"

namespace libgemm {

bool grouped_ring_takes_fp8(const GroupedArgs& a) { return routed::grouped_ring_fits<1>(a); }

hipError_t launch_grouped_ring_fp8(const GroupedArgs& a) {
    switch (a.fmt_a * 2 + a.fmt_b) {
        case 0: return a.b_kmajor ? routed::launch_grouped_ring<1, 0, 0, true>(a)
                                  : routed::launch_grouped_ring<1, 0, 0, false>(a);
        case 1: return a.b_kmajor ? routed::launch_grouped_ring<1, 0, 1, true>(a)
                                  : routed::launch_grouped_ring<1, 0, 1, false>(a);
        case 2: return a.b_kmajor ? routed::launch_grouped_ring<1, 1, 0, true>(a)
                                  : routed::launch_grouped_ring<1, 1, 0, false>(a);
        default: return a.b_kmajor ? routed::launch_grouped_ring<1, 1, 1, true>(a)
                                   : routed::launch_grouped_ring<1, 1, 1, false>(a);
    }
}

bool lora_ring_takes_fp8(const LoraArgs& a) { return ring::ring_fits<1, 64, true>(a, 64); }

hipError_t launch_lora_ring_fp8(const LoraArgs& a) {
    switch (a.fmt_a * 2 + a.fmt_b) {
        case 0: return routed::launch_lora_ring_any<1, 0, 0>(a);
        case 1: return routed::launch_lora_ring_any<1, 0, 1>(a);
        case 2: return routed::launch_lora_ring_any<1, 1, 0>(a);
        default: return routed::launch_lora_ring_any<1, 1, 1>(a);
    }
}

}  // namespace libgemm
