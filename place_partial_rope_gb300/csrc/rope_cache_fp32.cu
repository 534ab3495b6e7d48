// rope_cache_fp32.cu -- the cache kernels for dense rows of fp32.
#include "rope_cache_kernels.cuh"

namespace rope {

const void* cache_kernel_fp32(const CachePlan& p, bool write) {
    return write ? pick_cache<float, true>(p) : pick_cache<float, false>(p);
}

}  // namespace rope
