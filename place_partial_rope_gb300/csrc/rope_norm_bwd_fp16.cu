// rope_norm_bwd_fp16.cu -- norm and rotation of fp16 rows, backward.
#include "rope_norm_kernels.cuh"

namespace rope {

NormKernel norm_bwd_kernel_fp16(const NormPlan& p) {
    switch (p.chunks) {
        case 1: return norm_pick<__half, 1, true>(p);
        case 2: return norm_pick<__half, 2, true>(p);
        case 3: return norm_pick<__half, 3, true>(p);
        case 4: return norm_pick<__half, 4, true>(p);
        default: return NormKernel{nullptr, 0};
    }
}

}  // namespace rope
