// rope_latent_launch.cu -- kernel choice, grid, workspace and launches of the attention
// over latent rows.
#include <cuda.h>
#include <cuda_runtime.h>

#include "rope_latent.h"

namespace rope {
namespace {

TreeKernel kernel_of(const LatentPlan& p) {
    switch (p.store) {
        case ROPE_CACHE_BF16: return latent_kernel_bf16(p);
        case ROPE_CACHE_FP16: return latent_kernel_fp16(p);
        case ROPE_CACHE_FP8: return latent_kernel_fp8(p);
        default: return latent_kernel_int8(p);
    }
}

}  // namespace

// Tiles as narrow as the query rows allow.  Tensor copies where eights of rows lie in one
// page (and there is one: a map has no dim of 0) and rows are whole chunks: chunks of prompts in
// pages of 16 rows 396 us, and 504 in pages of 10, copied by threads.
// 8-bit rows pass through registers anyway.
LatentPlan choose_latent(int store, int64_t rows, int64_t k_dim, int64_t pages, int64_t page_size) {
    LatentPlan p{};
    p.store = store;
    p.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    p.boxes = (store == ROPE_CACHE_BF16 || store == ROPE_CACHE_FP16) && pages > 0 && page_size % 8 == 0 &&
              k_dim % 64 == 0;
    return p;
}

rope_status_t latent_blocks(const LatentPlan& p, int sm_count, int* blocks, const char** err) {
    if (sm_count > 0) {
        *blocks = sm_count;
        return ROPE_OK;
    }
    return tree_resident(kernel_of(p), blocks, err);
}

int64_t latent_workspace(const LatentPlan& p, int blocks) {
    const int64_t rows = int64_t(2) * blocks * p.rows;
    return rows * kLatentValues * int64_t(sizeof(float)) + rows * int64_t(sizeof(float2)) +
           int64_t(blocks) * int64_t(sizeof(TreeMeta));
}

rope_status_t launch_latent(const LatentPlan& p, const TreeArgs& args, void* workspace, int blocks,
                            rope_stream_t stream, const char** err) {
    const TreeKernel k = kernel_of(p);
    TreeArgs a = args;
    // Where a request's row tiles come in pairs (128 heads, say), so do blocks: two walk the two
    // row tiles of a pair in step, and what one brings from memory the other finds in L2:
    // 64 requests of 128 heads over 90 to 12000 bf16 rows 161 us, and 177 without.
    const int per = a.G % (2 * p.rows) == 0 && blocks % 2 == 0 ? 2 : 1;
    a.share = a.G / per;
    const int64_t rows = int64_t(2) * blocks * p.rows;
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part + rows * kLatentValues);
    a.meta = reinterpret_cast<TreeMeta*>(a.part_ml + rows);
    LatentMaps maps{};
    if (p.boxes) {
        a.box = 8;
        while (a.box < kLatentKeys && a.page_size % (2 * a.box) == 0) a.box *= 2;
        rope_status_t st = tree_map_eights(&maps.four, a, 4, err);
        if (st == ROPE_OK && latent_groups(a) > latent_value_groups(a)) st = tree_map_eights(&maps.one, a, 1, err);
        if (st != ROPE_OK) return st;
    }
    void* params[] = {&a, &maps};
    const rope_status_t st = tree_launch(k.main, blocks / per, per, k.threads, k.smem, params, stream, err);
    if (st != ROPE_OK || blocks / per < 2) return st;
    void* join[] = {&a};
    return tree_launch(k.join, blocks / per - 1, p.rows / 16 * 2 * per, kLatentJoinThreads, 0, join, stream, err);
}

}  // namespace rope
