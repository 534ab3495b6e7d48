// rope_axes.h -- what the host hands to the kernels of the positions call
// with several axes.  Not part of the public ABI.
#pragma once
#include "rope_internal.h"
#include "rope_serving.h"

namespace rope {

// Kernel parameter: each pair's frequency (omega = hi + lo, as in FreqTable)
// and axis, and where the axes' positions lie.  4.6 KB, staged into shared
// memory by every block.
struct AxisTable {
    float hi[kMaxPairs];
    float lo[kMaxPairs];
    uint8_t axis[kMaxPairs];
    int64_t pos_a;  // elements between axes
    int32_t axes;
};

const void* axes_kernel_bf16(const Plan& p);
const void* axes_kernel_fp16(const Plan& p);
const void* axes_kernel_fp32(const Plan& p);

// Launch one piece of an axes call (rope_axes_launch.cu).
rope_status_t launch_axes_piece(const Plan& plan, const KernelArgs& args, const AxisTable& table,
                                uint32_t blocks, rope_stream_t stream, const char** err);

}  // namespace rope
