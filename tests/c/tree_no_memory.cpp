// Host check of the kernel queries when host memory runs out: an error
// status, no exception (the callers are C).  The CUDA runtime is a stand-in:
// linked with the objects of rope_tree_launch.cu and rope_launch.cu, and without
// the runtime.
#include <new>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <cuda_runtime_api.h>

#include "rope_internal.h"
#include "rope_tree.h"

static bool g_full = false;

void* operator new(size_t n) {
    void* p = g_full ? nullptr : malloc(n);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void* p) noexcept { free(p); }
void operator delete(void* p, size_t) noexcept { free(p); }

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t) { return *n = 2, cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
    memset(a, 0, sizeof *a);
    return a->numRegs = 128, cudaSuccess;
}
const char* cudaGetErrorString(cudaError_t) { return "stand-in"; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return cudaSuccess; }
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes*, const void*) { return cudaErrorUnknown; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void**, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult*) {
    return cudaErrorUnknown;
}
}

extern "C" {
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
}

namespace rope {
static const char g_what[8] = "";
static TreeKernel kernel(int i) { return TreeKernel{g_what + i, g_what + i, 0, 128, 64, 0.0f, 0}; }
TreeKernel narrow_kernel_bf16(const TreePlan&) { return kernel(0); }
TreeKernel narrow_kernel_fp16(const TreePlan&) { return kernel(1); }
TreeKernel narrow_kernel_fp8(const TreePlan&) { return kernel(2); }
TreeKernel narrow_kernel_int8(const TreePlan&) { return kernel(3); }
TreeKernel tile_kernel_bf16(const TreePlan&) { return kernel(4); }
TreeKernel tile_kernel_fp16(const TreePlan&) { return kernel(5); }
TreeKernel tile_kernel_fp8(const TreePlan&) { return kernel(6); }
TreeKernel tile_kernel_int8(const TreePlan&) { return kernel(7); }
const void* kernel_for_bf16(const Plan&) { return g_what; }
const void* kernel_for_fp16(const Plan&) { return g_what; }
const void* kernel_for_fp32(const Plan&) { return g_what; }
}  // namespace rope

int main() {
    rope::TreePlan p{ROPE_BF16, ROPE_CACHE_BF16, 64, 64, 16};
    const char* err = "";
    int blocks = 0;
    try {
        g_full = true;
        const rope_status_t st = rope::tree_blocks(p, 0, &blocks, &err);
        g_full = false;
        printf("without memory: status %d (%s)\n", int(st), err);
        if (st != ROPE_ERR_CUDA || !strstr(err, "memory")) return 1;
        if (rope::tree_blocks(p, 0, &blocks, &err) != ROPE_OK || blocks != 304) return 1;
        g_full = true;  // what is known by now needs none
        if (rope::tree_blocks(p, 0, &blocks, &err) != ROPE_OK || blocks != 304) return 1;
        rope::Plan q{};
        int n = 0;
        if (rope::kernel_blocks_per_sm(q, &n, &err) != ROPE_ERR_CUDA || !strstr(err, "memory")) return 1;
        g_full = false;
        if (rope::kernel_blocks_per_sm(q, &n, &err) != ROPE_OK || n != 2) return 1;
    } catch (...) {
        g_full = false;
        printf("an exception reached the caller\n");
        return 1;
    }
    printf("ok\n");
    return 0;
}
