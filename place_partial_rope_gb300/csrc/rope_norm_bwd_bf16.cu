// rope_norm_bwd_bf16.cu -- norm and rotation of bf16 rows, backward.
#include "rope_norm_kernels.cuh"

namespace rope {

NormKernel norm_bwd_kernel_bf16(const NormPlan& p) {
    switch (p.chunks) {
        case 1: return norm_pick<__nv_bfloat16, 1, true>(p);
        case 2: return norm_pick<__nv_bfloat16, 2, true>(p);
        case 3: return norm_pick<__nv_bfloat16, 3, true>(p);
        case 4: return norm_pick<__nv_bfloat16, 4, true>(p);
        default: return NormKernel{nullptr, 0};
    }
}

}  // namespace rope
