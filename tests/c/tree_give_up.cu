// Device check of what the attention's tile kernel does when one of its waits
// gives up.  Every wait here has its limit, as in the library.
//
//   agree   threads of a role ask for the next run while `dead` is set and the
//           run is written down at about the same time: all of them take it or
//           none does.
//   fetch   the fetching warp with nobody to empty the rings: it gives up after
//           some seconds, and what it has fetched by then is left as it is.
//   call    whole calls without the thread that issues the products, or without
//           the softmax, in every second block: they end, and the results that
//           those blocks had a share in are NaN, joined ones too; the others
//           are right.
//
// Prints "ok ..." or what differed.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "rope_tree_launch.cu"
#include "rope_tree_tile.cuh"

// The kernel that launch_tree() and tree_blocks() get, whatever the plan.
static rope::TreeKernel g_kernel;

namespace rope {
TreeKernel narrow_kernel_bf16(const TreePlan&) { return g_kernel; }
TreeKernel narrow_kernel_fp16(const TreePlan&) { return g_kernel; }
TreeKernel narrow_kernel_fp8(const TreePlan&) { return g_kernel; }
TreeKernel narrow_kernel_int8(const TreePlan&) { return g_kernel; }
TreeKernel tile_kernel_bf16(const TreePlan&) { return g_kernel; }
TreeKernel tile_kernel_fp16(const TreePlan&) { return g_kernel; }
TreeKernel tile_kernel_fp8(const TreePlan&) { return g_kernel; }
TreeKernel tile_kernel_int8(const TreePlan&) { return g_kernel; }
}  // namespace rope

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
            sync.beat = 0;
        }
        __syncthreads();
        if (tid < 256) {
            pause((hash(seed ^ 55u) & 511u) + (hash(seed + uint32_t(tid) / 32) & 127u));
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

// ---------------------------------------------------------------- a small call

// R requests of one token and LEN rows each, one key head, 64 lanes, pages of 64
// rows in order; key codes of tile t (128 rows) are 1 + t, values' 65 + t.
template <class C, int R, int LEN>
struct Call {
    static constexpr int E = C::kWide ? 2 : 1, PAGES = R * LEN / 64, ELEMS = PAGES * 64 * 64;
    static_assert(LEN % 128 == 0, "whole tiles");
    TreePlan p{C::BF16 ? ROPE_BF16 : ROPE_FP16, C::STORE, 64, 64, C::ROWS};
    TreeArgs a{};
    int blocks = 0;
    char* ws = nullptr;

    template <class T>
    int make(bool several) {
        using K = TreeKernel;
        g_kernel = K{reinterpret_cast<const void*>(&rope_tree_tile_kernel<T>),
                     reinterpret_cast<const void*>(&rope_tree_join_kernel<C::ROWS, 64>), C::SMEM, kTileThreads, C::TN,
                     C::kBias, 256 * 192 + 256 * 64};
        const char* err = "";
        // (also: a kernel whose launch lacks the registers that it shares out is refused here)
        if (tree_blocks(p, 0, &blocks, &err) != ROPE_OK) {
            printf("FAIL %s\n", err);
            return 1;
        }
        if (!several) blocks = 1;
        char* codes[2];
        static char host[ELEMS * 2];
        for (int v = 0; v < 2; ++v) {
            for (int i = 0; i < ELEMS; ++i) {
                const int code = 1 + 64 * v + i / 64 % LEN / 128;
                if (E == 1) host[i] = char(code);
                else host[2 * i] = char(code), host[2 * i + 1] = 0;
            }
            CHECK(cudaMalloc(&codes[v], ELEMS * E));
            CHECK(cudaMemcpy(codes[v], host, ELEMS * E, cudaMemcpyHostToDevice));
        }
        static int32_t table[PAGES], start[R + 1], len[R];
        static float ones[PAGES * 64];
        for (int i = 0; i < PAGES; ++i) table[i] = i;
        for (int r = 0; r <= R; ++r) start[r] = r;
        for (int r = 0; r < R; ++r) len[r] = LEN;
        for (float& x : ones) x = 1.0f;
        void *dt, *ds, *dl, *ones_at, *q, *out, *lse;
        CHECK(cudaMalloc(&dt, sizeof table));
        CHECK(cudaMalloc(&ds, sizeof start));
        CHECK(cudaMalloc(&dl, sizeof len));
        CHECK(cudaMalloc(&ones_at, sizeof ones));
        CHECK(cudaMalloc(&q, R * 128));
        CHECK(cudaMalloc(&out, R * 128));
        CHECK(cudaMalloc(&lse, R * 4));
        CHECK(cudaMalloc(&ws, tree_workspace(p, blocks)));
        CHECK(cudaMemcpy(dt, table, sizeof table, cudaMemcpyHostToDevice));
        CHECK(cudaMemcpy(ds, start, sizeof start, cudaMemcpyHostToDevice));
        CHECK(cudaMemcpy(dl, len, sizeof len, cudaMemcpyHostToDevice));
        CHECK(cudaMemcpy(ones_at, ones, sizeof ones, cudaMemcpyHostToDevice));
        CHECK(cudaMemset(q, 0, R * 128));
        CHECK(cudaMemset(out, 0, R * 128));
        CHECK(cudaMemset(lse, 0, R * 4));
        CHECK(cudaMemset(ws, 0, tree_workspace(p, blocks)));
        a.k = codes[0];
        a.v = codes[1];
        a.ks = a.vs = C::kWide ? nullptr : static_cast<float*>(ones_at);
        for (int64_t* st : {a.k_st, a.v_st}) st[0] = 64 * 64 * E, st[1] = 64 * E, st[2] = 64 * E;
        for (int64_t* st : {a.ks_st, a.vs_st}) st[0] = 64, st[1] = 1, st[2] = 1;
        a.q = static_cast<char*>(q);
        a.out = static_cast<char*>(out);
        a.lse = static_cast<float*>(lse);
        a.q_st[0] = a.q_st[1] = a.o_st[0] = a.o_st[1] = 128;
        a.q_start = static_cast<int32_t*>(ds);
        a.kv_len = static_cast<int32_t*>(dl);
        a.table = static_cast<int32_t*>(dt);
        a.table_stride = LEN / 64;
        a.R = a.Tq = R;
        a.Hk = a.G = a.Hq = 1;
        a.Dk = a.Dv = 64;
        a.pages = PAGES;
        a.page_size = 64;
        a.max_len = LEN;
        a.div_page = FastDiv::make(64);
        a.div_group = FastDiv::make(1);
        a.scale_log2 = 0.125f;
        a.bf16 = C::BF16;
        return 0;
    }

    int launch() {
        const char* err = "";
        if (launch_tree(p, a, ws, blocks, nullptr, &err) != ROPE_OK) {
            printf("FAIL %s\n", err);
            return 1;
        }
        CHECK(cudaDeviceSynchronize());
        return 0;
    }
};

// ---------------------------------------------------------------- fetch

struct Seen {
    uint32_t dead;
    char smem[232448];
};
__device__ Seen g_seen;

// Nobody but the fetching warp, which shows what is in shared memory at its end.
template <class C>
struct FetchAlone : Tile<C> {
    __device__ void softmax(int) const {}
    __device__ void products() const {}
    __device__ void mend_tiles(int) const {}
    template <bool VALUES>
    __device__ void widen_tiles(int) const {}
    __device__ void fetches(const Place& place, const CUtensorMap* km, const CUtensorMap* vm) const {
        Tile<C>::fetches(place, km, vm);
        for (int i = int(threadIdx.x) % 32; i < C::RAW_AT + C::RAWS * C::RAW; i += 32) g_seen.smem[i] = this->smem[i];
        g_seen.dead = this->sync->dead;
    }
};

// The rings hold the first tiles: keys and values of as many as there are
// places, and not a byte of the next one.
template <class C>
static int fetch_alone(const char* what) {
    constexpr int TILES = 6;
    static Call<C, 1, 128 * TILES> call;
    static Seen seen;
    if (call.template make<FetchAlone<C>>(false) || call.launch()) return 1;
    CHECK(cudaMemcpyFromSymbol(&seen, g_seen, sizeof seen));
    int wrong = 0;
    for (int v = 0; v < 2; ++v)
        for (int s = 0; s < (C::kWide ? C::SLOTS : C::RAWS / 2); ++s) {
            const int at = C::kWide ? (v ? C::V_AT : C::K_AT) + s * C::K_SLOT : C::RAW_AT + (2 * s + v) * C::RAW;
            const int code = 1 + 64 * v + s;
            for (int i = 0; i < 128 * 64 * call.E; ++i) wrong += seen.smem[at + i] != (call.E == 2 && i % 2 ? 0 : code);
        }
    printf("%s: gave up %u, bytes of another tile %d\n", what, seen.dead, wrong);
    return seen.dead != 1 || wrong != 0;
}

// ---------------------------------------------------------------- call

template <class C>
struct NoProducts : Tile<C> {
    __device__ void products() const {
        if (blockIdx.x % 2 == 0) Tile<C>::products();
    }
};

template <class C>
struct NoSoftmax : Tile<C> {
    __device__ void softmax(int w) const {
        if (blockIdx.x % 2 == 0) Tile<C>::softmax(w);
    }
};

// Queries are zeros, so a result is the mean of the values: whole where the
// request's tiles are all in even blocks, and NaN where one is in an odd block.
template <class T, class C>
static int whole_calls(const char* what, bool fails) {
    constexpr int R = 40, TILES = 7;
    static Call<C, R, 128 * TILES> call;
    if (call.template make<T>(true)) return 1;
    // 8 units a block and 7 a request: some requests lie in one block, some in two
    call.blocks = 36;
    if (call.launch()) return 1;
    static uint16_t out[R][64];
    static float lse[R];
    CHECK(cudaMemcpy(out, call.a.out, sizeof out, cudaMemcpyDeviceToHost));
    CHECK(cudaMemcpy(lse, call.a.lse, sizeof lse, cudaMemcpyDeviceToHost));
    const int chunk = (R * TILES + call.blocks - 1) / call.blocks;  // (so few units a block count no leads)
    int wrong = 0, given_up = 0;
    for (int r = 0; r < R; ++r) {
        bool odd = false;
        for (int u = r * TILES; u < (r + 1) * TILES; ++u) odd = odd || u / chunk % 2 == 1;
        const bool none = odd && fails;
        given_up += none;
        wrong += none ? !(lse[r] != lse[r]) : !(lse[r] > 6.7 && lse[r] < 6.9);  // log 896
        for (int c = 0; c < 64; ++c) {
            const bool nan = C::BF16 ? (out[r][c] & 0x7fff) > 0x7f80 : (out[r][c] & 0x7fff) > 0x7c00;
            wrong += nan != none;
        }
    }
    printf("%s: %d of %d requests given up, %d numbers wrong\n", what, given_up, R, wrong);
    return wrong != 0 || (fails && (given_up == 0 || given_up == R));
}

template <class C>
static int whole_calls_of(const char* what) {
    printf("%s\n", what);
    return whole_calls<Tile<C>, C>("all roles", false) | whole_calls<NoProducts<C>, C>("without products", true) |
           whole_calls<NoSoftmax<C>, C>("without softmax", true);
}

int main(int argc, char** argv) {
    const char* mode = argc > 1 ? argv[1] : "";
    int bad = 1;
    if (!strcmp(mode, "agree")) bad = agree<1, 256>("groups") | agree<2, 192>("helpers") | agree<0, 32>("a warp");
    if (!strcmp(mode, "fetch"))
        bad = fetch_alone<TileCfg<ROPE_CACHE_BF16, 64, 64, 64>>("bf16") |
              fetch_alone<TileCfg<ROPE_CACHE_FP8, 64, 64, 64>>("fp8");
    if (!strcmp(mode, "call"))
        bad = whole_calls_of<TileCfg<ROPE_CACHE_BF16, 64, 64, 64>>("bf16") |
              whole_calls_of<TileCfg<ROPE_CACHE_FP8, 64, 64, 64>>("fp8") |
              whole_calls_of<TileCfg<ROPE_CACHE_BF16, 64, 64, 256>>("bf16, pairs") |
              whole_calls_of<TileCfg<ROPE_CACHE_FP8, 64, 64, 256>>("fp8, pairs");
    printf(bad ? "FAIL\n" : "ok\n");
    return bad;
}
