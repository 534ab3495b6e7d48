// rope_cache_bf16.cu -- the cache kernels for dense rows of bf16.
#include "rope_cache_kernels.cuh"

namespace rope {

const void* cache_kernel_bf16(const CachePlan& p, bool write) {
    return write ? pick_cache<__nv_bfloat16, true>(p) : pick_cache<__nv_bfloat16, false>(p);
}

}  // namespace rope
