// Products with bias, activation and residual, deep-ring kernel: FP8.
#include "bias_act_ring_impl.h"

namespace libgemm {

hipError_t launch_bias_act_ring_fp8(const BiasActArgs& a, int shape) {
    if (a.b_kmajor) {
        switch (a.fmt_a * 2 + a.fmt_b) {
            case 0: return bias_act::launch_ring_shape<1, 0, 0, true>(a, shape);
            case 1: return bias_act::launch_ring_shape<1, 0, 1, true>(a, shape);
            case 2: return bias_act::launch_ring_shape<1, 1, 0, true>(a, shape);
            default: return bias_act::launch_ring_shape<1, 1, 1, true>(a, shape);
        }
    }
    switch (a.fmt_a * 2 + a.fmt_b) {
        case 0: return bias_act::launch_ring_shape<1, 0, 0, false>(a, shape);
        case 1: return bias_act::launch_ring_shape<1, 0, 1, false>(a, shape);
        case 2: return bias_act::launch_ring_shape<1, 1, 0, false>(a, shape);
        default: return bias_act::launch_ring_shape<1, 1, 1, false>(a, shape);
    }
}

}  // namespace libgemm
