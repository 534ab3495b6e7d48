// rope_tile_bf16.cu -- the attention kernels over bf16 caches, for more query
// rows a key head.
#include "rope_tree_tile.cuh"

namespace rope {

TreeKernel tile_kernel_bf16(const TreePlan& p) {
    if (p.dk == 64) return pick_tile_rows<ROPE_CACHE_BF16, 64, 64>(p);
    if (p.dk == 128) return pick_tile_rows<ROPE_CACHE_BF16, 128, 128>(p);
    return pick_tile_rows<ROPE_CACHE_BF16, 192, 128>(p);
}

}  // namespace rope
