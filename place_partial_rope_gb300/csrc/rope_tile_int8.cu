// rope_tile_int8.cu -- the attention kernels over int8 caches, for more query
// rows a key head.
#include "rope_tree_tile.cuh"

namespace rope {

TreeKernel tile_kernel_int8(const TreePlan& p) {
    if (p.dk == 64) return pick_tile_rows<ROPE_CACHE_INT8, 64, 64>(p);
    if (p.dk == 128) return pick_tile_rows<ROPE_CACHE_INT8, 128, 128>(p);
    return pick_tile_rows<ROPE_CACHE_INT8, 192, 128>(p);
}

}  // namespace rope
