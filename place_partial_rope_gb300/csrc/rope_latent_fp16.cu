// rope_latent_fp16.cu -- the attention kernels over latent rows of fp16.
#include "rope_latent.cuh"

namespace rope {

TreeKernel latent_kernel_fp16(const LatentPlan& p) { return latent_pick<ROPE_CACHE_FP16>(p); }

}  // namespace rope
