// Device check of what the attention's tile kernel does when one of its waits
// gives up.  Every wait here has its limit, as in the library.
//
//   agree   threads of a role ask for the next run while `dead` is set and the
//           run is written down at about the same time: all of them take it or
//           none does.
//
// Prints "ok ..." or what differed.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "rope_tree_tile.cuh"

using namespace rope;

#define CHECK(x)                                                                \
    do {                                                                        \
        const cudaError_t e_ = (x);                                             \
        if (e_ != cudaSuccess) {                                                \
            printf("FAIL %s: %s\n", #x, cudaGetErrorString(e_));                \
            return 1;                                                           \
        }                                                                       \
    } while (0)

// ---------------------------------------------------------------- agree

__device__ uint32_t hash(uint32_t x) {
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    x *= 0x846ca68bu;
    return x ^ x >> 16;
}

__device__ void pause(uint32_t cycles) {
    const long long t = clock64();
    while (clock64() - t < cycles) {
    }
}

// 256 threads of a role (the first `asking` of them) and one more warp, which
// sets `dead` and, soon after, writes run 0 down.
template <int ID, int N>
__global__ void agree_kernel(const TreeArgs a, int rounds, unsigned* took, unsigned* differ) {
    using C = TileCfg<ROPE_CACHE_FP8, 64, 64, 64>;
    __shared__ TileSync sync;
    __shared__ uint32_t answer[256];
    const Tile<C> tile{a, nullptr, &sync, 0};
    const int tid = int(threadIdx.x);
    for (int i = 0; i < rounds; ++i) {
        const uint32_t seed = hash(blockIdx.x * 65537u + uint32_t(i));
        if (tid == 0) {
            sync.dead = 0;
            sync.runs = 0;
            sync.last = ~0u;
        }
        __syncthreads();
        if (tid < 256) {
            pause(hash(seed + uint32_t(tid) / 32) & 255u);
            RunAt x;
            if (tid < N || ID == 0) answer[tid] = tile.template take_all<ID, N>(0, x);
        } else if (tid == 256) {
            pause(hash(seed ^ 77u) & 255u);
            sync.dead = 1;
            pause(hash(seed ^ 99u) & 63u);
            sync.run[0] = RunAt{};
            __threadfence_block();
            sync.runs = 1;
        }
        __syncthreads();
        if (tid < (ID == 0 ? 256 : N)) {
            const int first = ID == 0 ? tid / 32 * 32 : 0;
            if (answer[tid] != answer[first]) atomicAdd(differ, 1u);
            else if (tid == first) atomicAdd(took + answer[tid], 1u);
        }
        __syncthreads();
    }
}

template <int ID, int N>
static int agree(const char* what) {
    unsigned* n;
    CHECK(cudaMalloc(&n, 12));
    CHECK(cudaMemset(n, 0, 12));
    agree_kernel<ID, N><<<64, 288>>>(TreeArgs{}, 500, n, n + 2);
    CHECK(cudaGetLastError());
    unsigned h[3];
    CHECK(cudaMemcpy(h, n, 12, cudaMemcpyDeviceToHost));
    CHECK(cudaFree(n));
    printf("%s: %u left together, %u went on together, %u apart\n", what, h[0], h[1], h[2]);
    return h[2] != 0 || h[0] == 0 || h[1] == 0;
}

int main(int argc, char** argv) {
    const char* mode = argc > 1 ? argv[1] : "";
    int bad = 1;
    if (!strcmp(mode, "agree")) bad = agree<1, 256>("groups") | agree<2, 192>("helpers") | agree<0, 32>("a warp");
    printf(bad ? "FAIL\n" : "ok\n");
    return bad;
}
