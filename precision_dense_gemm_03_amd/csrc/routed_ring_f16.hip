// Grouped and adapter products on the deep-ring kernel: FP16.
#include "routed_ring_impl.h"

namespace libgemm {

bool grouped_ring_takes_f16(const GroupedArgs& a) { return routed::grouped_ring_fits<2>(a); }

hipError_t launch_grouped_ring_f16(const GroupedArgs& a) {
    return a.b_kmajor ? routed::launch_grouped_ring<2, 0, 0, true>(a) : routed::launch_grouped_ring<2, 0, 0, false>(a);
}

bool lora_ring_takes_f16(const LoraArgs& a) { return ring::ring_fits<2, 64, true>(a, 64); }

hipError_t launch_lora_ring_f16(const LoraArgs& a) { return routed::launch_lora_ring_any<2, 0, 0>(a); }

}  // namespace libgemm
