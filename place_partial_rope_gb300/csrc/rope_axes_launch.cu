// rope_axes_launch.cu -- the launch of the positions call with several axes.
#include <cuda_runtime.h>

#include "rope_axes.h"

namespace rope {

rope_status_t launch_axes_piece(const Plan& plan, const KernelArgs& args, const AxisTable& table,
                                uint32_t blocks, rope_stream_t stream, const char** err) {
    const void* f = plan.dtype == ROPE_BF16   ? axes_kernel_bf16(plan)
                    : plan.dtype == ROPE_FP16 ? axes_kernel_fp16(plan)
                                              : axes_kernel_fp32(plan);
    if (!f) {
        *err = "internal error: no kernel instance for this plan";
        return ROPE_ERR_CUDA;
    }
    if (blocks == 0) return ROPE_OK;
    void* params[] = {const_cast<KernelArgs*>(&args), const_cast<AxisTable*>(&table)};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelExC(&cfg, f, params);
    if (e != cudaSuccess) {
        *err = cudaGetErrorString(e);
        (void)cudaGetLastError();
        return ROPE_ERR_CUDA;
    }
    return ROPE_OK;
}

}  // namespace rope
