// rope_axes_fp32.cu -- the fp32 instances of rope_partial_axes_kernel.
#include "rope_axes_kernels.cuh"

namespace rope {

const void* axes_kernel_fp32(const Plan& p) { return pick_axes<float>(p); }

}  // namespace rope
