// rope_norm_fwd_fp16.cu -- norm and rotation of fp16 rows, forward.
#include "rope_norm_kernels.cuh"

namespace rope {

NormKernel norm_fwd_kernel_fp16(const NormPlan& p) {
    switch (p.chunks) {
        case 1: return norm_pick<__half, 1, false>(p);
        case 2: return norm_pick<__half, 2, false>(p);
        case 3: return norm_pick<__half, 3, false>(p);
        case 4: return norm_pick<__half, 4, false>(p);
        default: return NormKernel{nullptr, 0};
    }
}

}  // namespace rope
