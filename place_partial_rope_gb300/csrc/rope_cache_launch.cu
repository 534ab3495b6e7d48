// rope_cache_launch.cu -- the launches of the cache kernels.
#include "rope_cache_kernels.cuh"

namespace rope {
namespace {

rope_status_t launch(const CachePlan& plan, const CacheArgs& args, bool write, rope_stream_t stream,
                     const char** err) {
    const void* f = plan.dtype == ROPE_BF16   ? cache_kernel_bf16(plan, write)
                    : plan.dtype == ROPE_FP16 ? cache_kernel_fp16(plan, write)
                                              : cache_kernel_fp32(plan, write);
    if (!f) {
        *err = "internal error: no kernel instance for this plan";
        return ROPE_ERR_CUDA;
    }
    const uint64_t threads = uint64_t(args.rows) * plan.lanes;
    void* params[] = {const_cast<CacheArgs*>(&args)};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((threads + kCacheThreads - 1) / kCacheThreads));
    cfg.blockDim = dim3(kCacheThreads);
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

}  // namespace

rope_status_t launch_cache_write(const CachePlan& plan, const CacheArgs& args, rope_stream_t stream,
                                 const char** err) {
    return launch(plan, args, true, stream, err);
}

rope_status_t launch_cache_read(const CachePlan& plan, const CacheArgs& args, rope_stream_t stream,
                                const char** err) {
    return launch(plan, args, false, stream, err);
}

}  // namespace rope
