// rope_latent.h -- what the host hands to the kernels of the attention over latent rows.
// Not part of the public ABI.  Arguments, division of the work and joining parts are
// those of rope_tree.h, with one key head, and values that are the keys' first lanes.
#pragma once
#include <cuda.h>

#include "rope_tree.h"

namespace rope {

constexpr int kLatentKeys = 64;      // cache rows of a tile
constexpr int kLatentLanes = 576;    // of a row, at most
constexpr int kLatentValues = 512;   // of those that are the value, at most
constexpr int kLatentThreads = 480;
constexpr int kLatentJoinThreads = 256;

struct LatentPlan {
    int store;  // rope_cache_dtype_t
    int rows;   // query rows of a tile: 16, 32 or 64
    bool boxes; // 16-bit rows of whole chunks, fetched by tensor copies: pages of a multiple of 8 rows
};

// Chunks of 64 lanes of a row; those of the values by two, a product each.
__host__ __device__ inline int latent_chunks(const TreeArgs& a) { return (a.Dk + 63) / 64; }
__host__ __device__ inline int latent_value_tiles(const TreeArgs& a) { return (a.Dv + 127) / 128; }
// Groups of a tile's chunks that come and go together: four chunks (the lanes of two value
// tiles), then those that hold no value's.  (Groups of 128 lanes: a wait more for each, of
// some 100 cycles, for products that take 256.)
__host__ __device__ inline int latent_value_groups(const TreeArgs& a) { return (a.Dv + 255) / 256; }
__host__ __device__ inline int latent_groups(const TreeArgs& a) {
    return latent_value_groups(a) + (latent_chunks(a) > 4 * latent_value_groups(a) ? 1 : 0);
}

// Tensor maps: four chunks a copy, and one.
struct LatentMaps {
    CUtensorMap four, one;
};

TreeKernel latent_kernel_bf16(const LatentPlan& p);
TreeKernel latent_kernel_fp16(const LatentPlan& p);
TreeKernel latent_kernel_fp8(const LatentPlan& p);
TreeKernel latent_kernel_int8(const LatentPlan& p);

// The kernel for `rows` query rows a request and pages of `page_size` rows of `k_dim` lanes.
LatentPlan choose_latent(int store, int64_t rows, int64_t k_dim, int64_t pages, int64_t page_size);

// The grid: one block an SM of the device (sm_count 0: the current one's).
rope_status_t latent_blocks(const LatentPlan& p, int sm_count, int* blocks, const char** err);

int64_t latent_workspace(const LatentPlan& p, int blocks);

rope_status_t launch_latent(const LatentPlan& p, const TreeArgs& args, void* workspace, int blocks,
                            rope_stream_t stream, const char** err);

}  // namespace rope
