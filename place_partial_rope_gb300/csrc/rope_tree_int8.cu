// rope_tree_int8.cu -- the attention kernels over int8 caches.
#include "rope_tree_kernels.cuh"

namespace rope {

TreeKernel tree_kernel_int8(const TreePlan& p) { return pick_tree<ROPE_CACHE_INT8>(p); }

}  // namespace rope
