// rope_tree_bf16.cu -- the attention kernels over bf16 caches, for up to 16 query
// rows a key head (and rows of 256 lanes).
#include "rope_tree_narrow.cuh"

namespace rope {

TreeKernel narrow_kernel_bf16(const TreePlan& p) {
    if (p.dk == 64) return narrow_kernel<ROPE_CACHE_BF16, 64, 64>();
    if (p.dk == 128) return narrow_kernel<ROPE_CACHE_BF16, 128, 128>();
    if (p.dk == 192) return narrow_kernel<ROPE_CACHE_BF16, 192, 128>();
    return narrow_kernel<ROPE_CACHE_BF16, 256, 256>();
}

}  // namespace rope
