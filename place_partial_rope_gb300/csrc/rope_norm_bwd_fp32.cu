// rope_norm_bwd_fp32.cu -- norm and rotation of fp32 rows, backward.
#include "rope_norm_kernels.cuh"

namespace rope {

NormKernel norm_bwd_kernel_fp32(const NormPlan& p) {
    switch (p.chunks) {
        case 1: return norm_pick<float, 1, true>(p);
        case 2: return norm_pick<float, 2, true>(p);
        case 3: return norm_pick<float, 3, true>(p);
        case 5: return norm_pick<float, 5, true>(p);
        case 8: return norm_pick<float, 8, true>(p);
        default: return NormKernel{nullptr, 0};
    }
}

}  // namespace rope
