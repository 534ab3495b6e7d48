// rope_tree.h -- what the host hands to the attention kernels.  Not part of
// the public ABI.
#pragma once
#include <stdint.h>
#include <vector_types.h>

#include "fast_div.h"
#include "rope_serving.h"

namespace rope {

constexpr int kNarrowThreads = 128;
constexpr int kTileThreads = 512;
constexpr int kJoinThreads = 256;

struct TreeArgs {
    const char* k;
    const char* v;
    const float* ks;  // scales of an 8-bit cache
    const float* vs;
    int64_t k_st[3], v_st[3];    // bytes: page, token, head
    int64_t ks_st[3], vs_st[3];  // elements
    const char* q;
    char* out;
    float* lse;                  // (Tq, Hq) or null
    int64_t q_st[2], o_st[2];    // bytes: token, head
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
    int64_t table_stride;
    const int64_t* tree;         // (Tq, words) or null: a chain
    float* part;                 // partial results: (2 * blocks, rows, DV)
    float2* part_ml;             // and their maxima and sums: (2 * blocks, rows)
    struct TreeMeta* meta;       // one per block
    int32_t words;
    int32_t R, Tq, Hk, G, Hq, Dk, Dv;
    int32_t pages, page_size, max_len;
    int32_t box;                 // tile kernels: rows of a fetch, a power of two that divides page_size
    FastDiv div_page, div_group;
    float scale_log2;            // scale * log2(e)
    bool bf16;                   // type of q and out (the cache's own for 16 bits)
};

// The group of row tiles that a block's first unit lies in, when it began in
// an earlier block (nt > 0): written by the block, read by the join kernel.
struct TreeMeta {
    int64_t u0;     // the unit of the group's first tile
    int64_t chunk;  // units per block
    int32_t r, h, m, nt, lead;
};

struct TreePlan {
    int dtype;    // rope_dtype_t of q
    int store;    // rope_cache_dtype_t
    int dk, dv;   // row lengths the kernel is built for (>= the call's)
    int rows;     // query rows of a tile: 16 (narrow kernel), 64, 128 or 256 (tile kernel)
};

// The kernel for rows of Dk and Dv, `rows` query rows a key head and `pages` pages
// of `page_size` rows, `tiles` cache tiles of which the page table has room for.
void choose_tree(int Dk, int Dv, int64_t rows, int64_t pages, int64_t page_size, int64_t tiles, TreePlan* p);

// The grid of a plan: the blocks that are resident on the device (sm_count
// 0), or an upper bound of that for a device of sm_count SMs.
rope_status_t tree_blocks(const TreePlan& p, int sm_count, int* blocks, const char** err);

int64_t tree_workspace(const TreePlan& p, int blocks);

rope_status_t launch_tree(const TreePlan& p, const TreeArgs& args, void* workspace, int blocks,
                          rope_stream_t stream, const char** err);

// A plan's kernels, and what their launch needs.
struct TreeKernel {
    const void* main;
    const void* join;
    int smem, threads;
    int tile;  // cache rows of a tile
    float bias;
    int regs;  // registers of a block that its warps share out among them; 0: they do not
};

// defined in rope_tree_*.cu (up to 16 query rows) and rope_tile_*.cu
TreeKernel narrow_kernel_bf16(const TreePlan& p);
TreeKernel narrow_kernel_fp16(const TreePlan& p);
TreeKernel narrow_kernel_fp8(const TreePlan& p);
TreeKernel narrow_kernel_int8(const TreePlan& p);
TreeKernel tile_kernel_bf16(const TreePlan& p);
TreeKernel tile_kernel_fp16(const TreePlan& p);
TreeKernel tile_kernel_fp8(const TreePlan& p);
TreeKernel tile_kernel_int8(const TreePlan& p);

}  // namespace rope
