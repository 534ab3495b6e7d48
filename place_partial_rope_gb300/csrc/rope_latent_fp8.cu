// rope_latent_fp8.cu -- the attention kernels over latent rows of fp8.
#include "rope_latent.cuh"

namespace rope {

TreeKernel latent_kernel_fp8(const LatentPlan& p) { return latent_pick<ROPE_CACHE_FP8>(p); }

}  // namespace rope
