// rope_pages.cu -- pages, slots and positions of a batch's new tokens, and pages given
// back.
//
// Mathematics: prefix sums over the requests of their tokens and of the pages that
// they need (or give back).  With them every token knows its request, place and
// page by itself: page p of a request that held h pages is entry p of its table row
// when p < h, and otherwise lies (pages needed by earlier requests) + p - h below the
// top of the stack; the same sums, page by page, give the table's new entries.
//
// What bounds it: latency; there is little to read and 12 bytes a token to write.
// So it is one launch of one cluster of up to 8 blocks, without a
// workspace.  Each block forms the sums of all requests for itself, a chunk of
// requests after the other, in shared memory; the cluster's barrier stands
// between the last read of a chunk's lengths and the first block's writing them in
// place; then the blocks share out the chunk's tokens (pages), four in a row a
// thread, which looks its first token's request up by halving.  Where there are places for
// many tokens, 8 blocks are too few to write them: a grid without clusters fills them in
// and leaves the lengths, and a launch after it writes those.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "rope_kernels.cuh"
#include "rope_pages.h"

namespace rope {
namespace {

namespace cg = cooperative_groups;

constexpr int kEach = 2;  // requests of a thread, in a chunk

// Sums over a block's threads of two numbers each: what comes before a thread's own, and
// all.  `scratch` holds 2 x (THREADS / 32) numbers.
template <int THREADS>
__device__ __forceinline__ void block_sums(int64_t a, int64_t b, int64_t* scratch, int64_t& before_a, int64_t& before_b,
                                           int64_t& all_a, int64_t& all_b) {
    constexpr int WARPS = THREADS / 32;
    const int lane = int(threadIdx.x) & 31, warp = int(threadIdx.x) >> 5;
    int64_t x = a, y = b;  // inclusive over the warp
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
        if (lane >= d) x += u, y += v;
    }
    __syncthreads();  // scratch has been read
    if (lane == 31) scratch[warp] = x, scratch[WARPS + warp] = y;
    __syncthreads();
    // every warp adds the warps' sums up for itself
    const int64_t wa = lane < WARPS ? scratch[lane] : 0, wb = lane < WARPS ? scratch[WARPS + lane] : 0;
    int64_t sa = wa, sb = wb;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t u = __shfl_up_sync(0xffffffffu, sa, d), v = __shfl_up_sync(0xffffffffu, sb, d);
        if (lane >= d) sa += u, sb += v;
    }
    all_a = __shfl_sync(0xffffffffu, sa, 31);
    all_b = __shfl_sync(0xffffffffu, sb, 31);
    before_a = __shfl_sync(0xffffffffu, sa - wa, warp) + x - a;
    before_b = __shfl_sync(0xffffffffu, sb - wb, warp) + y - b;
}

// The last k in [0, n) with from[k] <= at; from[0] <= at.
__device__ __forceinline__ int find(const int64_t* from, int n, int64_t at) {
    int lo = 0;
    for (int step = n; step > 1;) {
        step = (step + 1) / 2;
        if (lo + step < n && from[lo + step] <= at) lo += step;
    }
    return lo;
}

// Pages that hold `len` rows.
__device__ __forceinline__ int32_t pages_of(const PagesArgs& a, int32_t len) {
    return len <= 0 ? 0 : static_cast<int32_t>(a.div_page.div(uint32_t(len) - 1)) + 1;
}

__device__ __forceinline__ int32_t length(const PagesArgs& a, int r) { return min(max(a.kv_len[r], 0), a.max_len); }

// FILL: writes slots, positions and the table; STATE: lengths, offsets and the count.  Both: one
// cluster; FILL alone: any grid, which only reads what STATE changes.
template <int THREADS, bool FILL, bool STATE>
__global__ void __launch_bounds__(THREADS) rope_cache_grow_kernel(const __grid_constant__ PagesArgs a) {
    constexpr int CHUNK = THREADS * kEach;
    __shared__ int64_t start[CHUNK];  // tokens before a request
    __shared__ int64_t asked[CHUNK];  // pages needed before it
    __shared__ int32_t rows[CHUNK];   // its rows so far; ~rows: it is not granted
    __shared__ int64_t scratch[2 * (THREADS / 32)];
    cg::cluster_group cluster = cg::this_cluster();
    enter_after_predecessor();
    const int64_t rank = blockIdx.x;
    const int64_t me = rank * THREADS + threadIdx.x, threads = int64_t(gridDim.x) * THREADS;
    const int32_t count = min(max(*a.free_count, 0), a.capacity);
    int64_t tokens = 0, needed = 0;  // of the chunks before
    __shared__ int32_t went;         // pages that are granted: up to the last request that gets any
    if (threadIdx.x == 0) went = 0;
    for (int r0 = 0; r0 < a.R; r0 += CHUNK) {
        int32_t len[kEach], grown[kEach], need[kEach];
        int64_t n[kEach];
        bool ok[kEach];
        int64_t sum_n = 0, sum_need = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int r = r0 + int(threadIdx.x) * kEach + i;
            len[i] = grown[i] = need[i] = 0;
            n[i] = 0;
            ok[i] = false;
            if (r >= a.R) continue;
            len[i] = length(a, r);
            n[i] = max(__ldg(a.n + r), 0);
            ok[i] = len[i] + n[i] <= a.max_len;
            grown[i] = ok[i] ? len[i] + int32_t(n[i]) : len[i];
            need[i] = pages_of(a, grown[i]) - pages_of(a, len[i]);
            sum_n += n[i];
            sum_need += need[i];
        }
        int64_t bn, bp, all_n, all_p;
        block_sums<THREADS>(sum_n, sum_need, scratch, bn, bp, all_n, all_p);
        int32_t end = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int k = int(threadIdx.x) * kEach + i;
            ok[i] = ok[i] && (need[i] == 0 || needed + bp + need[i] <= count);
            start[k] = tokens + bn;
            asked[k] = needed + bp;
            rows[k] = ok[i] ? len[i] : ~len[i];
            if (ok[i] && need[i] > 0) end = int32_t(needed + bp + need[i]);  // <= count
            bn += n[i];
            bp += need[i];
        }
        end = __reduce_max_sync(0xffffffffu, end);
        if ((threadIdx.x & 31) == 0 && end > 0) atomicMax(&went, end);
        // all blocks have read the chunk's lengths (and the count), this block's sums are there
        if constexpr (FILL && STATE) cluster.sync();
        else __syncthreads();
        if (STATE && rank == 0) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int k = int(threadIdx.x) * kEach + i, r = r0 + k;
                if (r >= a.R) continue;
                a.kv_len[r] = ok[i] ? grown[i] : len[i];
                a.q_start[r] = int32_t(min(start[k], int64_t(0x7fffffff)));
                if (a.granted) a.granted[r] = ok[i] ? 1 : 0;
            }
        }
        const int here = min(CHUNK, a.R - r0);
        // slots and positions; tokens past the last place (of a request that is not granted there
        // may be any number) are not looked at
        const int64_t to = FILL ? min(tokens + all_n, a.T) : 0;
        for (int64_t t0 = tokens + me * 4; t0 < to; t0 += threads * 4) {
            int k = find(start, here, t0), page = -1;
            int32_t p = -1;
            for (int i = 0; i < 4 && t0 + i < to; ++i) {
                const int64_t t = t0 + i;
                while (k + 1 < here && start[k + 1] <= t) ++k, p = -1;
                const int32_t old = rows[k] < 0 ? ~rows[k] : rows[k];
                const int64_t at = old + (t - start[k]);
                int64_t slot = -1;
                if (rows[k] >= 0) {
                    uint32_t q, off;
                    a.div_page.divmod(uint32_t(at), q, off);
                    if (int32_t(q) != p) {
                        p = int32_t(q);
                        const int32_t held = pages_of(a, old);
                        page = p < held ? a.table[int64_t(r0 + k) * a.table_stride + p]
                                        : __ldg(a.free_pages + (count - 1 - (asked[k] + p - held)));
                    }
                    if (page >= 0) slot = int64_t(page) * a.div_page.d + off;
                }
                a.slots[t] = slot;
                if (a.positions) a.positions[t] = static_cast<int32_t>(min(at, int64_t(0x7fffffff)));
            }
        }
        // the table's new entries: granted pages are the first `count` that are asked for, but
        // for those of a request that gets only a part
        const int64_t last = FILL ? min(needed + all_p, int64_t(count)) : 0;
        for (int64_t e = needed + me; e < last; e += threads) {
            const int k = find(asked, here, e);
            if (rows[k] >= 0)
                a.table[int64_t(r0 + k) * a.table_stride + pages_of(a, rows[k]) + (e - asked[k])] =
                    __ldg(a.free_pages + (count - 1 - e));
        }
        tokens += all_n;
        needed += all_p;
        __syncthreads();  // the chunk's numbers have been read
    }
    if constexpr (FILL && STATE) cluster.sync();  // every block has read the count, also where there are no requests
    if (STATE && rank == 0 && threadIdx.x == 0) {
        a.q_start[a.R] = int32_t(min(tokens, int64_t(0x7fffffff)));
        *a.free_count = count - went;
    }
    for (int64_t t = tokens + me; FILL && t < a.T; t += threads) {
        a.slots[t] = -1;
        if (a.positions) a.positions[t] = 0;
    }
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) rope_cache_trim_kernel(const __grid_constant__ PagesArgs a) {
    constexpr int CHUNK = THREADS * kEach;
    __shared__ int64_t start[CHUNK];  // pages that go, before a request's
    __shared__ int32_t first[CHUNK];  // the first page of a request that goes
    __shared__ int64_t scratch[2 * (THREADS / 32)];
    cg::cluster_group cluster = cg::this_cluster();
    enter_after_predecessor();
    const int64_t rank = cluster.block_rank(), blocks = cluster.num_blocks();
    const int64_t me = rank * THREADS + threadIdx.x, threads = blocks * THREADS;
    const int32_t count = min(max(*a.free_count, 0), a.capacity);
    // how many go, of all requests
    int64_t mine = 0, total, none, zero, nil;
    for (int r = int(threadIdx.x); r < a.R; r += THREADS) {
        const int32_t len = length(a, r), keep = min(max(__ldg(a.n + r), 0), len);
        mine += pages_of(a, len) - pages_of(a, keep);
    }
    block_sums<THREADS>(mine, 0, scratch, none, zero, total, nil);
    int64_t gone = 0;
    for (int r0 = 0; r0 < a.R; r0 += CHUNK) {
        int32_t keep[kEach];
        int64_t sum = 0, n[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int k = int(threadIdx.x) * kEach + i, r = r0 + k;
            n[i] = 0;
            keep[i] = 0;
            first[k] = 0;
            if (r >= a.R) continue;
            const int32_t len = length(a, r);
            keep[i] = min(max(__ldg(a.n + r), 0), len);
            first[k] = pages_of(a, keep[i]);
            n[i] = pages_of(a, len) - first[k];
            sum += n[i];
        }
        int64_t before, all;
        block_sums<THREADS>(sum, 0, scratch, before, zero, all, nil);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            start[int(threadIdx.x) * kEach + i] = gone + before;
            before += n[i];
        }
        cluster.sync();  // all blocks have read the chunk's lengths, this block's sums are there
        if (rank == 0)
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int r = r0 + int(threadIdx.x) * kEach + i;
                if (r < a.R) a.kv_len[r] = keep[i];
            }
        const int here = min(CHUNK, a.R - r0);
        for (int64_t e = gone + me; e < gone + all; e += threads) {
            const int k = find(start, here, e);
            int32_t* entry = a.table + int64_t(r0 + k) * a.table_stride + first[k] + (e - start[k]);
            const int64_t place = count + total - 1 - e;
            if (place < a.capacity) a.free_pages[place] = *entry;
            *entry = -1;
        }
        gone += all;
        __syncthreads();  // the chunk's numbers have been read
    }
    cluster.sync();  // every block has read the count
    if (rank == 0 && threadIdx.x == 0)
        *a.free_count = static_cast<int32_t>(min(int64_t(count) + total, int64_t(a.capacity)));
}

rope_status_t failed(cudaError_t e, const char** err) {
    *err = cudaGetErrorString(e);
    (void)cudaGetLastError();
    return ROPE_ERR_CUDA;
}

rope_status_t launch(const void* f, int threads, int blocks, bool cluster, const PagesArgs& args,
                     rope_stream_t stream, const char** err) {
    void* params[] = {const_cast<PagesArgs*>(&args)};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelExC(&cfg, f, params);
    return e == cudaSuccess ? ROPE_OK : failed(e, err);
}

constexpr int kFew = 256, kMany = 1024;
constexpr int64_t kWide = 16384;

// Small batches: a block of 256 threads, whose sums take fewer steps.
bool few(const PagesArgs& a) { return a.R <= kFew * kEach && a.T <= 4 * kFew; }  // to grow

int blocks_for(int64_t work) {
    int b = 1;
    while (b < 8 && int64_t(b) * kMany * 4 < work) b *= 2;
    return b;
}

}  // namespace

// From 16384 places on a grid of up to one block an SM and two launches: 500000 tokens of 512
// requests grown and given back, copies of the table and the lengths between, 172 us with the one
// cluster and a trim of one block of 256, 50 us so.
rope_status_t launch_grow(const PagesArgs& args, rope_stream_t stream, const char** err) {
    if (few(args))
        return launch(reinterpret_cast<const void*>(&rope_cache_grow_kernel<kFew, true, true>), kFew, 1, true, args,
                      stream, err);
    if (args.T < kWide)
        return launch(reinterpret_cast<const void*>(&rope_cache_grow_kernel<kMany, true, true>), kMany,
                      blocks_for(args.T), true, args, stream, err);
    int device = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return failed(e, err);
    const int64_t blocks = (args.T + kMany * 4 - 1) / (kMany * 4);
    const rope_status_t st = launch(reinterpret_cast<const void*>(&rope_cache_grow_kernel<kMany, true, false>), kMany,
                                    static_cast<int>(blocks < sms ? blocks : sms), false, args, stream, err);
    if (st != ROPE_OK) return st;
    return launch(reinterpret_cast<const void*>(&rope_cache_grow_kernel<kMany, false, true>), kMany, 1, false, args,
                  stream, err);
}

// How many pages go is known on the device only (a few of a request that goes on, all of one that
// has ended), but the table bounds them, and the stack: up to 1024 one block of 256 threads, up
// to 65536 of one chunk of requests a cluster of 8, else 8 blocks of 1024.  A call that gives
// few pages back takes 2.7 to 3.6 us on 1 or 8 blocks of 256 and 1 us more on 1024, where the sums
// take longer; 262144 pages of 32 requests 560 us, 85 and 40; 16384 pages of two requests 37 us, 18 and 17.
rope_status_t launch_trim(const PagesArgs& args, rope_stream_t stream, const char** err) {
    const int64_t held = int64_t(args.R) * args.max_pages, most = held < args.capacity ? held : args.capacity;
    if (args.R <= kFew * kEach && most <= 65536)
        return launch(reinterpret_cast<const void*>(&rope_cache_trim_kernel<kFew>), kFew, most <= 4 * kFew ? 1 : 8, true,
                      args, stream, err);
    return launch(reinterpret_cast<const void*>(&rope_cache_trim_kernel<kMany>), kMany, 8, true, args, stream, err);
}

}  // namespace rope
