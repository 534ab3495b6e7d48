// rope_tree_bf16.cu -- the attention kernels over bf16 caches.
#include "rope_tree_kernels.cuh"

namespace rope {

TreeKernel tree_kernel_bf16(const TreePlan& p) { return pick_tree<ROPE_CACHE_BF16>(p); }

}  // namespace rope
