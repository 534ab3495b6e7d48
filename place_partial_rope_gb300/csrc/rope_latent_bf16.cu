// rope_latent_bf16.cu -- the attention kernels over latent rows of bf16.
#include "rope_latent.cuh"

namespace rope {

TreeKernel latent_kernel_bf16(const LatentPlan& p) { return latent_pick<ROPE_CACHE_BF16>(p); }

}  // namespace rope
