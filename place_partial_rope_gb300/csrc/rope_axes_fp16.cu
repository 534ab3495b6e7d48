// rope_axes_fp16.cu -- the fp16 instances of rope_partial_axes_kernel.
#include "rope_axes_kernels.cuh"

namespace rope {

const void* axes_kernel_fp16(const Plan& p) { return pick_axes<__half>(p); }

}  // namespace rope
