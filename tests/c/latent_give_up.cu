// Device check of what the attention over latent rows does when its waits give up.
// Every wait here has its limit, as in the library.
//
// Whole calls, with all roles, and without one of them (the scores' or the values' products,
// the softmax, the helpers) in every second block: they end, and the results that
// those blocks had a share in are NaN, joined ones too; the others are right.
//
// Prints "ok" or what differed.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "rope_latent.cuh"
#include "rope_latent_launch.cu"
#include "rope_tree_launch.cu"

// The kernel that launch_latent() and latent_blocks() get, whatever the plan.
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
TreeKernel latent_kernel_bf16(const LatentPlan&) { return g_kernel; }
TreeKernel latent_kernel_fp16(const LatentPlan&) { return g_kernel; }
TreeKernel latent_kernel_fp8(const LatentPlan&) { return g_kernel; }
TreeKernel latent_kernel_int8(const LatentPlan&) { return g_kernel; }
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

template <class C>
struct NoScores : Latent<C> {
    __device__ void scores() const {
        if (blockIdx.x % 2 == 0) Latent<C>::scores();
    }
};

template <class C>
struct NoProducts : Latent<C> {
    __device__ void products() const {
        if (blockIdx.x % 2 == 0) Latent<C>::products();
    }
};

template <class C>
struct NoSoftmax : Latent<C> {
    __device__ void softmax(int group) const {
        if (blockIdx.x % 2 == 0) Latent<C>::softmax(group);
    }
};

template <class C>
struct NoHelpers : Latent<C> {
    __device__ void help(int id) const {
        if (blockIdx.x % 2 == 0) Latent<C>::help(id);
    }
};

// R requests of one token, ROWS heads and the same LEN rows of ones each, in pages of 64.
constexpr int R = 40, TILES = 7, LEN = 64 * TILES, DK = 576, DV = 512;

template <class C>
struct Call {
    static constexpr int E = C::kWide ? 2 : 1, HQ = C::ROWS;
    LatentPlan p{C::STORE, C::ROWS, C::BOXES};
    TreeArgs a{};
    void *q, *out, *lse, *ws, *cache, *ones, *table, *start, *len;
    // 8 units a block (7.8, too few for leads) and 7 a request: some requests lie in one block, some in two
    static constexpr int BLOCKS = 36;

    int make() {
        const int n = LEN * DK;
        static uint16_t host[LEN * DK];
        const int one = C::BF16 ? 0x3f80 : C::kWide ? 0x3c00 : C::STORE == ROPE_CACHE_FP8 ? 0x3838 : 0x0101;
        for (int i = 0; i < n; ++i) host[i] = uint16_t(one);
        static float scale[LEN];
        static int32_t pages[R * TILES], starts[R + 1], lens[R];
        for (float& x : scale) x = 1.0f;
        for (int i = 0; i < R * TILES; ++i) pages[i] = i % TILES;
        for (int r = 0; r <= R; ++r) starts[r] = r;
        for (int& x : lens) x = LEN;
        const struct { void** to; const void* from; size_t bytes; } all[] = {
            {&cache, host, size_t(n) * E}, {&ones, scale, sizeof scale},      {&table, pages, sizeof pages},
            {&start, starts, sizeof starts}, {&len, lens, sizeof lens},       {&q, nullptr, size_t(R) * HQ * DK * 2},
            {&out, nullptr, size_t(R) * HQ * DV * 2}, {&lse, nullptr, size_t(R) * HQ * 4},
            {&ws, nullptr, size_t(latent_workspace(p, BLOCKS))}};
        for (const auto& x : all) {
            CHECK(cudaMalloc(x.to, x.bytes));
            if (x.from) CHECK(cudaMemcpy(*x.to, x.from, x.bytes, cudaMemcpyHostToDevice));
        }
        a.k = a.v = static_cast<char*>(cache);
        a.ks = a.vs = static_cast<float*>(ones);
        for (int64_t* st : {a.k_st, a.v_st}) st[0] = 64 * DK * E, st[1] = st[2] = DK * E;
        for (int64_t* st : {a.ks_st, a.vs_st}) st[0] = 64, st[1] = st[2] = 1;
        a.q = static_cast<char*>(q);
        a.out = static_cast<char*>(out);
        a.lse = static_cast<float*>(lse);
        a.q_st[0] = HQ * DK * 2, a.q_st[1] = DK * 2;
        a.o_st[0] = HQ * DV * 2, a.o_st[1] = DV * 2;
        a.q_start = static_cast<int32_t*>(start);
        a.kv_len = static_cast<int32_t*>(len);
        a.table = static_cast<int32_t*>(table);
        a.table_stride = TILES;
        a.R = a.Tq = R;
        a.Hk = 1;
        a.G = a.Hq = HQ;
        a.Dk = DK;
        a.Dv = DV;
        a.pages = TILES;
        a.page_size = 64;
        a.max_len = LEN;
        a.div_page = FastDiv::make(64);
        a.div_group = FastDiv::make(HQ);
        a.scale_log2 = 0.125f;
        a.bf16 = C::BF16;
        return 0;
    }

    template <class T>
    int run(const char* what, bool fails) {
        g_kernel = latent_of<T>();
        const char* err = "";
        int resident = 0;  // (asked for: it allows the kernel its shared memory)
        CHECK(cudaMemset(q, 0, size_t(R) * HQ * DK * 2));
        CHECK(cudaMemset(out, 0, size_t(R) * HQ * DV * 2));
        CHECK(cudaMemset(lse, 0, size_t(R) * HQ * 4));
        CHECK(cudaMemset(ws, 0, latent_workspace(p, BLOCKS)));
        if (latent_blocks(p, 0, &resident, &err) != ROPE_OK || resident < BLOCKS ||
            launch_latent(p, a, ws, BLOCKS, nullptr, &err) != ROPE_OK) {
            printf("FAIL %s\n", err);
            return 1;
        }
        CHECK(cudaDeviceSynchronize());
        static uint16_t o[R][HQ][DV];
        static float l[R][HQ];
        CHECK(cudaMemcpy(o, out, sizeof o, cudaMemcpyDeviceToHost));
        CHECK(cudaMemcpy(l, lse, sizeof l, cudaMemcpyDeviceToHost));
        const int chunk = (R * TILES + BLOCKS - 1) / BLOCKS, one = C::BF16 ? 0x3f80 : 0x3c00;
        int wrong = 0, given_up = 0;
        for (int r = 0; r < R; ++r) {
            bool odd = false;
            for (int u = r * TILES; u < (r + 1) * TILES; ++u) odd = odd || u / chunk % 2 == 1;
            const bool none = odd && fails;
            given_up += none;
            for (int h = 0; h < HQ; ++h) {
                wrong += none ? !(l[r][h] != l[r][h]) : !(l[r][h] > 6.104f && l[r][h] < 6.106f);  // log 448
                for (int c = 0; c < DV; ++c) {
                    const bool nan = (o[r][h][c] & 0x7fff) > (C::BF16 ? 0x7f80 : 0x7c00);
                    wrong += none ? !nan : o[r][h][c] != one;
                }
            }
        }
        printf("%s: %d of %d requests given up, %d numbers wrong\n", what, given_up, R, wrong);
        return wrong != 0 || (fails && (given_up == 0 || given_up == R));
    }
};

template <int STORE, int ROWS, bool BOXES>
static int calls() {
    using C = LatentCfg<STORE, ROWS, BOXES>;
    static Call<C> call;
    if (call.make()) return 1;
    int bad = call.template run<Latent<C>>("all roles", false);
    if (!bad) bad = call.template run<NoScores<C>>("without scores", true);
    if (!bad) bad = call.template run<NoProducts<C>>("without products", true);
    if (!bad) bad = call.template run<NoSoftmax<C>>("without softmax", true);
    if (!bad) bad = call.template run<NoHelpers<C>>("without helpers", true);
    return bad;
}

int main(int argc, char** argv) {
    const char* mode = argc > 1 ? argv[1] : "";
    int bad = 1;
    if (!strcmp(mode, "boxes")) bad = calls<ROPE_CACHE_BF16, 64, true>();
    if (!strcmp(mode, "rows")) bad = calls<ROPE_CACHE_FP16, 32, false>();
    if (!strcmp(mode, "codes")) bad = calls<ROPE_CACHE_FP8, 16, false>();
    printf(bad ? "FAIL\n" : "ok\n");
    return bad;
}
