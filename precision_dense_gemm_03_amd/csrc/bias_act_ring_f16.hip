// Products with bias, activation and residual, deep-ring kernel: FP16.
#include "bias_act_ring_impl.h"

namespace libgemm {

bool bias_act_ring_takes(int kind, const BiasActArgs& a) {
    if (kind == KIND_F16) return a.b_kmajor ? ring::ring_fits<2, 64, true>(a, 64) : ring::ring_fits<2, 64, false>(a, 64);
    return a.b_kmajor ? ring::ring_fits<1, 64, true>(a, 64) : ring::ring_fits<1, 64, false>(a, 64);
}

hipError_t launch_bias_act_ring_f16(const BiasActArgs& a, int shape) {
    return a.b_kmajor ? bias_act::launch_ring_shape<2, 0, 0, true>(a, shape)
                      : bias_act::launch_ring_shape<2, 0, 0, false>(a, shape);
}

}  // namespace libgemm
