// rope_norm_fwd_fp32.cu -- norm and rotation of fp32 rows, forward.
#include "rope_norm_kernels.cuh"

namespace rope {

NormKernel norm_fwd_kernel_fp32(const NormPlan& p) {
    switch (p.chunks) {
        case 1: return norm_pick<float, 1, false>(p);
        case 2: return norm_pick<float, 2, false>(p);
        case 3: return norm_pick<float, 3, false>(p);
        case 5: return norm_pick<float, 5, false>(p);
        case 8: return norm_pick<float, 8, false>(p);
        default: return NormKernel{nullptr, 0};
    }
}

}  // namespace rope
