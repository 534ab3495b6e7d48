// rope_tree_fp8.cu -- the attention kernels over fp8 caches.
#include "rope_tree_kernels.cuh"

namespace rope {

TreeKernel tree_kernel_fp8(const TreePlan& p) { return pick_tree<ROPE_CACHE_FP8>(p); }

}  // namespace rope
