// rope_tree_launch.cu -- kernel choice, grid, workspace and launches of the
// attention over the cache.
#include <mutex>
#include <unordered_map>

#include <cuda.h>

#include "rope_tree_common.cuh"

namespace rope {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kBlocksPerSm = 8;  // no kernel here has more resident blocks an SM

struct Resident {
    int sms, per_sm;
};

std::mutex g_mu;
std::unordered_map<const void*, Resident> g_resident[kMaxDevices];

TreeKernel kernel_of(const TreePlan& p) {
    const bool narrow = p.rows == 16;
    switch (p.store) {
        case ROPE_CACHE_BF16: return narrow ? narrow_kernel_bf16(p) : tile_kernel_bf16(p);
        case ROPE_CACHE_FP16: return narrow ? narrow_kernel_fp16(p) : tile_kernel_fp16(p);
        case ROPE_CACHE_FP8: return narrow ? narrow_kernel_fp8(p) : tile_kernel_fp8(p);
        default: return narrow ? narrow_kernel_int8(p) : tile_kernel_int8(p);
    }
}

rope_status_t cuda_fail(cudaError_t e, const char** err) {
    *err = cudaGetErrorString(e);
    (void)cudaGetLastError();
    return ROPE_ERR_CUDA;
}

// The kernel's resident blocks on device `dev`, under the lock.
rope_status_t resident_on(int dev, const TreeKernel& k, Resident* out, const char** err) {
    auto it = g_resident[dev].find(k.main);
    if (it != g_resident[dev].end()) {
        *out = it->second;
        return ROPE_OK;
    }
    Resident r{};
    cudaError_t e = cudaFuncSetAttribute(k.main, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&r.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&r.per_sm, k.main, k.threads, k.smem);
    cudaFuncAttributes at{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, k.main);
    if (e != cudaSuccess) return cuda_fail(e, err);
    if (at.numRegs * k.threads < k.regs) {  // a share that is not there would be waited for
        *err = "the attention kernel was built with too few registers";
        return ROPE_ERR_CUDA;
    }
    if (r.per_sm < 1) {
        *err = "the attention kernel does not fit this device";
        return ROPE_ERR_CUDA;
    }
    if (r.per_sm > kBlocksPerSm) r.per_sm = kBlocksPerSm;
    g_resident[dev][k.main] = r;
    *out = r;
    return ROPE_OK;
}

// The kernel's resident blocks on the current device; the first call for a
// device and kernel also allows its shared memory.
rope_status_t resident(const TreeKernel& k, Resident* out, const char** err) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, err);
    if (dev < 0 || dev >= kMaxDevices) {
        *err = "device number out of range";
        return ROPE_ERR_CUDA;
    }
    try {
        std::lock_guard<std::mutex> lk(g_mu);
        return resident_on(dev, k, out, err);
    } catch (...) {  // the callers are C
        *err = "out of host memory";
        return ROPE_ERR_CUDA;
    }
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                            CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
    static const Encode f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<Encode>(p);
    }();
    return f;
}

// The map of a cache tensor: (lane, head, token of the page, page).  `lanes`
// are those of a fetch: 64 of a 16-bit row, in the 128-byte swizzle, or a whole
// row of codes.
rope_status_t map_of(CUtensorMap* map, const void* base, int dim, const TreeArgs& a, const int64_t* st, bool wide,
                     int lanes, const char** err) {
    const Encode encode = encoder();
    if (!encode) {
        *err = "the driver has no cuTensorMapEncodeTiled";
        return ROPE_ERR_CUDA;
    }
    // the stride of a dim of one is not looked at by the call: any valid one does
    const cuuint64_t sizes[4] = {cuuint64_t(dim), cuuint64_t(a.Hk), cuuint64_t(a.page_size), cuuint64_t(a.pages)};
    const cuuint64_t strides[3] = {a.Hk > 1 ? cuuint64_t(st[2]) : 16, a.page_size > 1 ? cuuint64_t(st[1]) : 16,
                                   a.pages > 1 ? cuuint64_t(st[0]) : 16};
    // L2 fetches no more than a head's row: with 256 bytes for fp8 rows of 128 the
    // neighbouring head's came along, and went before its turn (980 MB read for 618);
    // bf16 rows of 192 + 128, 32 requests of 8000 rows: 240 us, and 225 so
    const int row = dim * (wide ? 2 : 1);
    const CUtensorMapL2promotion promotion = row % 256 == 0   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                             : row % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                             : row % 64 == 0  ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                              : CU_TENSOR_MAP_L2_PROMOTION_NONE;
    const cuuint32_t box[4] = {cuuint32_t(lanes), 1, cuuint32_t(a.box), 1}, steps[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, wide ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
                              const_cast<void*>(base), sizes, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                              promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        *err = "the cache's sizes or strides do not fit a tensor map";
        return ROPE_ERR_CUDA;
    }
    return ROPE_OK;
}

rope_status_t launch(const void* f, dim3 grid, int threads, int smem, void** params,
                     rope_stream_t stream, const char** err) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelExC(&cfg, f, params);
    return e == cudaSuccess ? ROPE_OK : cuda_fail(e, err);
}

}  // namespace

// Which kernel: by types, row lengths, the query rows of a key head, and the cache
// tiles (128 rows of one key head) that the page table has room for.  Both sides
// of each border, in us (32 requests of 8000 rows, 8 key heads, 128 + 128 lanes
// unless it says otherwise):
//   16-bit, up to 16 query rows: narrow 201, 64-row tiles 175; 8 requests of 4096
//   rows 59 and 44.  But 4 requests of 4096 rows 28 and 32, and one of 4097 rows
//   with 2 key heads 13.3 and 13.8, the tile kernel's start being the longer one:
//   to 8 tiles an SM (of this card's 152), the narrow kernel.
//   fp8, up to 16 rows: narrow 176, 64-row tiles 193 (codes become fp16 in registers
//   there, in shared memory here).  32 rows: 323 and 189.
//   64 rows: 64-row tiles 182 (bf16) and 190 (fp8), 128-row tiles 185 and 210.
//   256 rows: a pair of tiles that share the cache's, 249 (bf16) and 522 (fp8);
//   128-row tiles, the cache read twice, 351 and 430, as fp8 pairs have room for
//   64-row cache tiles only; with 64-lane rows, which have room for more, 215
//   and 330 against 263 and 367; fp8 rows of 192 + 128, 612 and 625.
// Tensor copies take boxes of at least 8 rows of a page; pages that those do not
// divide, and rows of more than 192 lanes (whose O does not fit tensor memory
// twice), stay with the narrow kernel.  So does a cache without pages: a tensor
// map has no dim of 0.
void choose_tree(int Dk, int Dv, int64_t rows, int64_t pages, int64_t page_size, int64_t tiles, TreePlan* p) {
    constexpr int64_t kFewTiles = 8 * 152;  // (the plan is made without a device, too)
    if (Dk <= 64) p->dk = 64, p->dv = 64;
    else if (Dk <= 128) p->dk = 128, p->dv = 128;
    else if (Dk <= 192 && Dv <= 128) p->dk = 192, p->dv = 128;
    else p->dk = 256, p->dv = 256;
    const bool wide = p->store == ROPE_CACHE_BF16 || p->store == ROPE_CACHE_FP16;
    if (p->dk == 256 || pages == 0 || page_size % 8 || (rows <= 16 && (!wide || tiles <= kFewTiles)))
        p->rows = 16;
    else p->rows = rows <= 64 ? 64 : rows <= 128 || !(wide || p->dk == 64) ? 128 : 256;
}

rope_status_t tree_blocks(const TreePlan& p, int sm_count, int* blocks, const char** err) {
    if (sm_count > 0) {
        *blocks = sm_count * kBlocksPerSm;
        return ROPE_OK;
    }
    Resident r;
    const rope_status_t st = resident(kernel_of(p), &r, err);
    if (st == ROPE_OK) *blocks = r.sms * r.per_sm;
    return st;
}

rope_status_t tree_resident(const TreeKernel& k, int* blocks, const char** err) {
    Resident r;
    const rope_status_t st = resident(k, &r, err);
    if (st == ROPE_OK) *blocks = r.sms * r.per_sm;
    return st;
}

rope_status_t tree_map_eights(CUtensorMap* map, const TreeArgs& a, int pieces, const char** err) {
    const Encode encode = encoder();
    if (!encode) {
        *err = "the driver has no cuTensorMapEncodeTiled";
        return ROPE_ERR_CUDA;
    }
    const cuuint64_t row = cuuint64_t(a.k_st[1]);
    const cuuint64_t sizes[5] = {64, 8, cuuint64_t(a.Dk / 64), cuuint64_t(a.page_size / 8), cuuint64_t(a.pages)};
    const cuuint64_t strides[4] = {row, 128, row * 8, a.pages > 1 ? cuuint64_t(a.k_st[0]) : 16};
    const cuuint32_t box[5] = {64, 8, cuuint32_t(pieces), cuuint32_t(a.box / 8), 1}, steps[5] = {1, 1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, const_cast<char*>(a.k), sizes, strides, box,
                              steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        *err = "the cache's sizes or strides do not fit a tensor map";
        return ROPE_ERR_CUDA;
    }
    return ROPE_OK;
}

rope_status_t tree_launch(const void* f, int blocks, int per, int threads, int smem, void** params,
                          rope_stream_t stream, const char** err) {
    return launch(f, dim3(blocks, per), threads, smem, params, stream, err);
}

int64_t tree_workspace(const TreePlan& p, int blocks) {
    const int64_t rows = int64_t(2) * blocks * p.rows;
    return rows * p.dv * int64_t(sizeof(float)) + rows * int64_t(sizeof(float2)) +
           int64_t(blocks) * int64_t(sizeof(TreeMeta));
}

rope_status_t launch_tree(const TreePlan& p, const TreeArgs& args, void* workspace, int blocks,
                          rope_stream_t stream, const char** err) {
    const TreeKernel k = kernel_of(p);
    TreeArgs a = args;
    const int64_t rows = int64_t(2) * blocks * p.rows;
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part + rows * p.dv);
    a.meta = reinterpret_cast<TreeMeta*>(a.part_ml + rows);
    CUtensorMap km, vm;
    if (p.rows != 16) {
        const bool wide = p.store == ROPE_CACHE_BF16 || p.store == ROPE_CACHE_FP16;
        a.box = 8;
        while (a.page_size % (2 * a.box) == 0 && 2 * a.box <= k.tile) a.box *= 2;
        rope_status_t st = map_of(&km, a.k, a.Dk, a, a.k_st, wide, wide ? 64 : p.dk, err);
        if (st == ROPE_OK) st = map_of(&vm, a.v, a.Dv, a, a.v_st, wide, wide ? 64 : p.dv, err);
        if (st != ROPE_OK) return st;
    }
    void* params[] = {&a, &km, &vm};  // the narrow kernel takes the first
    rope_status_t st = launch(k.main, dim3(blocks), k.threads, k.smem, params, stream, err);
    if (st != ROPE_OK || blocks < 2) return st;
    float bias = k.bias;
    void* join[] = {&a, &bias};
    // tile kernels: few borders cut a group, which has pieces for many blocks
    return launch(k.join, dim3(blocks - 1, p.rows > 16 ? 4 : 1), kJoinThreads, 0, join, stream, err);
}

}  // namespace rope
