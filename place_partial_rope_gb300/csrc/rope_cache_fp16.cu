// rope_cache_fp16.cu -- the cache kernels for dense rows of fp16.
#include "rope_cache_kernels.cuh"

namespace rope {

const void* cache_kernel_fp16(const CachePlan& p, bool write) {
    return write ? pick_cache<__half, true>(p) : pick_cache<__half, false>(p);
}

}  // namespace rope
