// rope_tree_fp16.cu -- the attention kernels over fp16 caches.
#include "rope_tree_kernels.cuh"

namespace rope {

TreeKernel tree_kernel_fp16(const TreePlan& p) { return pick_tree<ROPE_CACHE_FP16>(p); }

}  // namespace rope
