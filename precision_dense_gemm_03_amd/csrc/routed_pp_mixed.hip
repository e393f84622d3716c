// Grouped and adapter products on the ping-pong tile kernel: the FP8 operand
// pairs with E5M2, in the tile heights that serve every size (192 rows; the
// pairs E4M3 x E4M3 and FP16 have the others too).
#include "routed_pp_impl.h"

namespace libgemm {

hipError_t launch_grouped_pp_mixed(const GroupedArgs& a) {
    switch (a.fmt_a * 2 + a.fmt_b) {
        case 1: return a.b_kmajor ? routed::launch_grouped_pp<1, 0, 1, true, 192, false>(a)
                                  : routed::launch_grouped_pp<1, 0, 1, false, 192, false>(a);
        case 2: return a.b_kmajor ? routed::launch_grouped_pp<1, 1, 0, true, 192, false>(a)
                                  : routed::launch_grouped_pp<1, 1, 0, false, 192, false>(a);
        default: return a.b_kmajor ? routed::launch_grouped_pp<1, 1, 1, true, 192, false>(a)
                                   : routed::launch_grouped_pp<1, 1, 1, false, 192, false>(a);
    }
}

hipError_t launch_lora_pp_mixed(const LoraArgs& a) {
    switch (a.fmt_a * 2 + a.fmt_b) {
        case 1: return routed::launch_lora_pp<1, 0, 1, 192>(a);
        case 2: return routed::launch_lora_pp<1, 1, 0, 192>(a);
        default: return routed::launch_lora_pp<1, 1, 1, 192>(a);
    }
}

}  // namespace libgemm
