// rope_norm_launch.cu -- kernel choice, grids and launches of the norm and rotation,
// and the kernel that adds up the parts of the weights' gradients.
#include <mutex>
#include <unordered_map>

#include "rope_kernels.cuh"
#include "rope_norm.h"

namespace rope {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kJoinRows = 32;

std::mutex g_mu;
std::unordered_map<const void*, int> g_resident[kMaxDevices];  // blocks an SM

rope_status_t cuda_fail(cudaError_t e, const char** err) {
    *err = cudaGetErrorString(e);
    (void)cudaGetLastError();
    return ROPE_ERR_CUDA;
}

rope_status_t launch(const void* f, dim3 grid, dim3 block, void** params, rope_stream_t stream, const char** err) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelExC(&cfg, f, params);
    return e == cudaSuccess ? ROPE_OK : cuda_fail(e, err);
}

// Sums of the blocks' rows of a side: 32 lanes a block, 32 threads a lane, which
// take the rows in turn and are added up in order.
__global__ void __launch_bounds__(kNormJoinLanes* kJoinRows)
    rope_norm_join_kernel(const __grid_constant__ NormJoin j) {
    __shared__ float sums[kJoinRows][kNormJoinLanes + 1];
    enter_after_predecessor();
    const float* part = j.part[blockIdx.y];
    if (!part) return;
    const int lane = int(blockIdx.x) * kNormJoinLanes + int(threadIdx.x);
    float s = 0.0f;
    if (lane < j.lanes)
#pragma unroll 8
        for (int b = int(threadIdx.y); b < j.blocks; b += kJoinRows) s += part[int64_t(b) * j.lanes + lane];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || lane >= j.lanes) return;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) s += sums[k][threadIdx.x];
    j.out[blockIdx.y][lane] = s;
}

}  // namespace

NormKernel norm_kernel(const NormPlan& p) {
    switch (p.dtype) {
        case ROPE_BF16: return p.back ? norm_bwd_kernel_bf16(p) : norm_fwd_kernel_bf16(p);
        case ROPE_FP16: return p.back ? norm_bwd_kernel_fp16(p) : norm_fwd_kernel_fp16(p);
        default: return p.back ? norm_bwd_kernel_fp32(p) : norm_fwd_kernel_fp32(p);
    }
}

rope_status_t launch_norm_fwd(const NormKernel& k, const NormArgs& args, rope_stream_t stream, const char** err) {
    const uint64_t items = uint64_t(args.side[0].items) + (args.sides == 2 ? args.side[1].items : 0);
    const uint64_t per = uint64_t(kNormThreads >> args.lanes_log2);
    // The kernel numbers items in 32 bits, those of both sides and the rest of the last block:
    // a side has less than 2^31, so all are at most 2^32, which `per`, a power of two, divides.
    static_assert((kNormThreads & (kNormThreads - 1)) == 0, "a block's items are a power of two");
    if ((items + per - 1) / per * per > uint64_t(1) << 32) {
        *err = "internal error: more rows than a launch can number";
        return ROPE_ERR_CUDA;
    }
    void* params[] = {const_cast<NormArgs*>(&args)};
    return launch(k.f, dim3(static_cast<unsigned>((items + per - 1) / per)), dim3(kNormThreads), params, stream, err);
}

rope_status_t norm_sm_count(int* sms, const char** err) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    return e == cudaSuccess ? ROPE_OK : cuda_fail(e, err);
}

rope_status_t norm_blocks(const NormKernel& k, const NormArgs& args, int* blocks, const char** err) {
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, err);
    if (dev < 0 || dev >= kMaxDevices) {
        *err = "device number out of range";
        return ROPE_ERR_CUDA;
    }
    try {
        std::lock_guard<std::mutex> lk(g_mu);
        auto it = g_resident[dev].find(k.f);
        if (it != g_resident[dev].end()) {
            per_sm = it->second;
        } else {
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k.f, kNormThreads, 0);
            if (e != cudaSuccess) return cuda_fail(e, err);
            if (per_sm < 1) per_sm = 1;
            if (per_sm > kNormBlocksPerSm) per_sm = kNormBlocksPerSm;
            g_resident[dev][k.f] = per_sm;
        }
    } catch (...) {  // the callers are C
        *err = "out of host memory";
        return ROPE_ERR_CUDA;
    }
    const uint32_t per = uint32_t(kNormThreads >> args.lanes_log2);
    uint32_t most = args.side[0].items;
    if (args.sides == 2 && args.side[1].items > most) most = args.side[1].items;
    const uint64_t wanted = (uint64_t(most) + per - 1) / per, room = uint64_t(sms) * per_sm;
    *blocks = static_cast<int>(wanted < room ? wanted : room);
    return ROPE_OK;
}

rope_status_t launch_norm_bwd(const NormKernel& k, const NormArgs& args, int blocks, rope_stream_t stream,
                              const char** err) {
    void* params[] = {const_cast<NormArgs*>(&args)};
    return launch(k.f, dim3(static_cast<unsigned>(blocks)), dim3(kNormThreads), params, stream, err);
}

rope_status_t launch_norm_join(const NormJoin& join, rope_stream_t stream, const char** err) {
    void* params[] = {const_cast<NormJoin*>(&join)};
    const unsigned x = static_cast<unsigned>((join.lanes + kNormJoinLanes - 1) / kNormJoinLanes);
    return launch(reinterpret_cast<const void*>(&rope_norm_join_kernel), dim3(x, 2), dim3(kNormJoinLanes, kJoinRows),
                  params, stream, err);
}

}  // namespace rope
