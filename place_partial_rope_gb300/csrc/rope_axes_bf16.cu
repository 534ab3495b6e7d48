// rope_axes_bf16.cu -- the bf16 instances of rope_partial_axes_kernel.
#include "rope_axes_kernels.cuh"

namespace rope {

const void* axes_kernel_bf16(const Plan& p) { return pick_axes<__nv_bfloat16>(p); }

}  // namespace rope
