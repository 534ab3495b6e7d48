// rope_norm_fwd_bf16.cu -- norm and rotation of bf16 rows, forward.
#include "rope_norm_kernels.cuh"

namespace rope {

NormKernel norm_fwd_kernel_bf16(const NormPlan& p) {
    switch (p.chunks) {
        case 1: return norm_pick<__nv_bfloat16, 1, false>(p);
        case 2: return norm_pick<__nv_bfloat16, 2, false>(p);
        case 3: return norm_pick<__nv_bfloat16, 3, false>(p);
        case 4: return norm_pick<__nv_bfloat16, 4, false>(p);
        default: return NormKernel{nullptr, 0};
    }
}

}  // namespace rope
