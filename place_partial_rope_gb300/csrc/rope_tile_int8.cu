// rope_tile_int8.cu -- the attention kernels over int8 caches, for more query
// rows a key head.
#include "rope_tree_tile.cuh"

namespace rope {

TreeKernel tile_kernel_int8(const TreePlan& p) {
    const bool pair = p.rows == 256;
    if (p.dk == 64) return pair ? tile_kernel<ROPE_CACHE_INT8, 64, 64, true>() : tile_kernel<ROPE_CACHE_INT8, 64, 64, false>();
    if (p.dk == 128)
        return pair ? tile_kernel<ROPE_CACHE_INT8, 128, 128, true>() : tile_kernel<ROPE_CACHE_INT8, 128, 128, false>();
    return pair ? tile_kernel<ROPE_CACHE_INT8, 192, 128, true>() : tile_kernel<ROPE_CACHE_INT8, 192, 128, false>();
}

}  // namespace rope
