// rope_norm.h -- what the host hands to the kernels of the norm and rotation.  Not
// part of the public ABI.
#pragma once
#include <stdint.h>

#include "fast_div.h"
#include "rope_step.h"

namespace rope {

constexpr int kNormThreads = 256;
constexpr int kNormBlocksPerSm = 8;   // no backward has more resident blocks an SM
constexpr int kNormJoinLanes = 32;    // lanes of the weights that a joining block adds up

// The queries' or the keys' rows of a launch.
struct NormRows {
    const char* x;
    char* out;
    const char* grad;
    const char* weight;
    float* rstd;
    float* part;  // backward: (blocks, normed lanes) sums of the weights' gradient, or null
    int64_t x_st[3], out_st[3], grad_st[3];  // bytes: batch, token, head
    int32_t heads;
    int32_t groups;  // of U heads
    uint32_t items;  // tokens x groups
    FastDiv div_groups;
};

struct NormArgs {
    NormRows side[2];
    const char* cos;
    const char* sin;
    int64_t cos_st[2], sin_st[2];  // bytes
    int32_t sides, D, n0, n1, start, end;
    int32_t lanes_log2;  // lanes of a warp that share a row
    bool weight32;       // weights are fp32
    bool wide;           // rows allow 16-byte accesses
    bool pairs_cs;       // cos and sin allow accesses of pairs (kTurnPairs)
    bool interleave;     // pairs are adjacent lanes
    float eps, inv_n;
    FastDiv div_S;
};

// How pairs lie: within a chunk of 16 bytes, which turns as a whole or not at all; within a
// chunk, each for itself; half-split, the partners of a chunk a whole chunk; anything
// else.  In all but the last, chunks are normed as a whole or not at all.
enum NormTurn : int { kTurnNear = 0, kTurnPairs = 1, kTurnFar = 2, kTurnAny = 3 };

struct NormPlan {
    int dtype;   // rope_dtype_t
    int turn;    // NormTurn
    int chunks;  // 16-byte chunks of a row that a lane holds
    bool many;   // several heads a thread
    bool back;
};

struct NormKernel {
    const void* f;
    int heads;  // heads a thread takes
};

NormKernel norm_fwd_kernel_bf16(const NormPlan& p);
NormKernel norm_fwd_kernel_fp16(const NormPlan& p);
NormKernel norm_fwd_kernel_fp32(const NormPlan& p);
NormKernel norm_bwd_kernel_bf16(const NormPlan& p);
NormKernel norm_bwd_kernel_fp16(const NormPlan& p);
NormKernel norm_bwd_kernel_fp32(const NormPlan& p);

NormKernel norm_kernel(const NormPlan& p);  // f is null: there is none

rope_status_t launch_norm_fwd(const NormKernel& k, const NormArgs& args, rope_stream_t stream, const char** err);

// The backward's grid: blocks that are resident on the current device, at most those
// that there is work for.
rope_status_t norm_blocks(const NormKernel& k, const NormArgs& args, int* blocks, const char** err);

rope_status_t launch_norm_bwd(const NormKernel& k, const NormArgs& args, int blocks, rope_stream_t stream,
                              const char** err);

// weight_grad = the sum of `blocks` rows of each side that wants one.
struct NormJoin {
    const float* part[2];
    float* out[2];
    int32_t lanes, blocks;
};

rope_status_t launch_norm_join(const NormJoin& join, rope_stream_t stream, const char** err);

rope_status_t norm_sm_count(int* sms, const char** err);

}  // namespace rope
