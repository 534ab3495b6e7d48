// rope_latent_int8.cu -- the attention kernels over latent rows of int8.
#include "rope_latent.cuh"

namespace rope {

TreeKernel latent_kernel_int8(const LatentPlan& p) { return latent_pick<ROPE_CACHE_INT8>(p); }

}  // namespace rope
