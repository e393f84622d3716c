// Products with bias, activation and residual, ping-pong tile kernel: the FP8
// operand pairs with E5M2 (192 rows).
#include "bias_act_pp_impl.h"

namespace libgemm {

hipError_t launch_bias_act_pp_mixed(const BiasActArgs& a) {
    switch (a.fmt_a * 2 + a.fmt_b) {
        case 1: return a.b_kmajor ? bias_act::launch_pp<1, 0, 1, true, 192>(a) : bias_act::launch_pp<1, 0, 1, false, 192>(a);
        case 2: return a.b_kmajor ? bias_act::launch_pp<1, 1, 0, true, 192>(a) : bias_act::launch_pp<1, 1, 0, false, 192>(a);
        default: return a.b_kmajor ? bias_act::launch_pp<1, 1, 1, true, 192>(a) : bias_act::launch_pp<1, 1, 1, false, 192>(a);
    }
}

}  // namespace libgemm
