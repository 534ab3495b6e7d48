// rope_tc.cuh -- the instructions that the kernels on tcgen05 share: barriers in shared
// memory, tensor memory, matrix descriptors and products.
#pragma once
#include "rope_f32x2.cuh"
#include "rope_tree_common.cuh"

namespace rope {

constexpr uint32_t kSpins = 1u << 20;  // tries of one wait before it gives up: 1.5 s and more
constexpr uint32_t kPolls = 1u << 26;  // looks of a thread that does not pause

__device__ __forceinline__ void bar_init(unsigned long long* b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(unsigned long long* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(b)) : "memory");
}

__device__ __forceinline__ bool bar_test(unsigned long long* b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(smem_addr(b)), "r"(parity)
                 : "memory");
    return ok != 0;
}

// Without the pause that try_wait may take: for a thread that looks at several.
__device__ __forceinline__ bool bar_poll(unsigned long long* b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(smem_addr(b)), "r"(parity)
                 : "memory");
    return ok != 0;
}

__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void to_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define ROPE_R8(r, i) "=f"(r[i]), "=f"(r[i + 1]), "=f"(r[i + 2]), "=f"(r[i + 3]), "=f"(r[i + 4]), "=f"(r[i + 5]), \
                      "=f"(r[i + 6]), "=f"(r[i + 7])
#define ROPE_B8(r, i) "+f"(r[i]), "+f"(r[i + 1]), "+f"(r[i + 2]), "+f"(r[i + 3]), "+f"(r[i + 4]), "+f"(r[i + 5]), \
                      "+f"(r[i + 6]), "+f"(r[i + 7])
#define ROPE_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
                      "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of the thread's lane.
__device__ __forceinline__ void tmem_ld32(float* r, uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : ROPE_R8(r, 0), ROPE_R8(r, 8), ROPE_R8(r, 16), ROPE_R8(r, 24)
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(float* r, uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : ROPE_R8(r, 0), ROPE_R8(r, 8)
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_here16(float* r) { asm volatile("" : ROPE_B8(r, 0), ROPE_B8(r, 8)); }

// After tmem_wait_ld: what was loaded is not touched before this.
__device__ __forceinline__ void tmem_here32(float* r) {
    asm volatile("" : ROPE_B8(r, 0), ROPE_B8(r, 8), ROPE_B8(r, 16), ROPE_B8(r, 24));
}

__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
        ROPE_W8(r, 0), ROPE_W8(r, 8), ROPE_W8(r, 16), ROPE_W8(r, 24)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(at),
        ROPE_W8(r, 0), ROPE_W8(r, 8)
        : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle.  Keys and queries: rows
// of 128 bytes along the sum, groups of eight rows 1024 bytes apart (`lead`
// unused).  Values: 64 columns a line, the next 64 `lead` bytes on, groups of
// eight cache rows 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_matrix(uint32_t at, uint32_t lead) {
    return uint64_t((at & 0x3ffffu) >> 4) | (uint64_t(lead >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// 128 x N, fp32 sums, both factors of the storage type's product type; B_MN:
// the second factor's columns are contiguous (values).
template <bool BF16, int N, bool B_MN>
__host__ __device__ constexpr uint32_t mma_shape() {
    return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((B_MN ? 1u : 0u) << 16) |
           (uint32_t(N / 8) << 17) | (uint32_t(128 / 16) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(shape), "r"(uint32_t(add))
                 : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
                 "r"(a), "l"(b), "r"(shape), "r"(uint32_t(add))
                 : "memory");
}

// The barrier gets an arrival when every product issued so far is done.
__device__ __forceinline__ void mma_commit(unsigned long long* b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(b))
                 : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

}  // namespace rope
