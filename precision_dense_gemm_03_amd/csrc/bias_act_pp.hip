// Products with bias, activation and residual, ping-pong tile kernel: FP16 and E4M3 x E4M3.
#include "bias_act_pp_impl.h"

namespace libgemm {

bool bias_act_pp_takes_f16(const BiasActArgs& a) { return bias_act::pp_takes<2>(a); }
bool bias_act_pp_takes_fp8(const BiasActArgs& a) { return bias_act::pp_takes<1>(a); }

hipError_t launch_bias_act_pp_f16(const BiasActArgs& a, int bm) {
    if (bm == 256) return a.b_kmajor ? bias_act::launch_pp<2, 0, 0, true, 256>(a) : bias_act::launch_pp<2, 0, 0, false, 256>(a);
    return a.b_kmajor ? bias_act::launch_pp<2, 0, 0, true, 192>(a) : bias_act::launch_pp<2, 0, 0, false, 192>(a);
}

hipError_t launch_bias_act_pp_e4m3(const BiasActArgs& a, int bm) {
    if (bm == 256) return a.b_kmajor ? bias_act::launch_pp<1, 0, 0, true, 256>(a) : bias_act::launch_pp<1, 0, 0, false, 256>(a);
    return a.b_kmajor ? bias_act::launch_pp<1, 0, 0, true, 192>(a) : bias_act::launch_pp<1, 0, 0, false, 192>(a);
}

}  // namespace libgemm
