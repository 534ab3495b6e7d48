// Device check of how the attention over latent rows divides its work among blocks.
//
// Every block walks its share and writes down its runs, nothing else.  On the host: each cache
// tile of each (request, row tile) lies in one run; a group that is cut has its parts in
// blocks that follow each other, at places of their own, and its later blocks' first
// run says so to the join; and no block has more to do than the others by more than a
// tile and a lead, a masked tile (one that drafted rows fill) counted as four.
//
// Prints "ok" or what differed.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "rope_tree_common.cuh"

using namespace rope;

#define CHECK(x)                                                                \
    do {                                                                        \
        const cudaError_t e_ = (x);                                             \
        if (e_ != cudaSuccess) {                                                \
            printf("FAIL %s: %s\n", #x, cudaGetErrorString(e_));                \
            return 1;                                                           \
        }                                                                       \
    } while (0)

constexpr int ROWS = 64, TN = 64, THREADS = 480, BLOCKS = 152;

struct Found {
    int r, m, t0, count;
    int64_t slot;
};

__global__ void __launch_bounds__(THREADS) divide(const __grid_constant__ TreeArgs a, Found* runs, int most, int* counts) {
    __shared__ int64_t scratch[THREADS / 16 + 2];
    const Place place = find_place<ROWS, TN, THREADS, true>(a, scratch);
    if (threadIdx.x != 0) return;
    LatentWalk walk = latent_walk_from<ROWS, TN>(a, place);
    RunAt x;
    int n = 0;
    TreeMeta meta{0, place.chunk, 0, 0, 0, 0, 0};
    while (next_run<ROWS, TN>(a, walk, x)) {
        if (n == 0) meta = meta_of(place, walk, x);
        if (n < most) runs[int64_t(blockIdx.x) * most + n] = Found{x.r, x.m, x.t0, x.count, x.slot};
        ++n;
    }
    counts[blockIdx.x] = n;
    a.meta[blockIdx.x] = meta;
}

static int check(const char* what, const std::vector<int>& n, const std::vector<int>& len, int heads) {
    const int R = int(n.size());
    std::vector<int32_t> starts(R + 1, 0);
    for (int r = 0; r < R; ++r) starts[r + 1] = starts[r] + n[r];
    std::vector<int64_t> first(R + 1, 0);  // groups before a request's
    auto tiles = [&](int r) { return std::max(1, (len[r] + TN - 1) / TN); };
    auto masked = [&](int r) { return std::min(n[r] / TN, tiles(r)); };
    int64_t all = 0;
    for (int r = 0; r < R; ++r) {
        first[r + 1] = first[r] + (int64_t(n[r]) * heads + ROWS - 1) / ROWS;
        all += (first[r + 1] - first[r]) * tiles(r);
    }
    const bool leads = all >= BLOCKS * 8;
    const int most = int(first[R] + 1);
    TreeArgs a{};
    int32_t *qs, *ln;
    Found* runs;
    int* counts;
    CHECK(cudaMalloc(&qs, (R + 1) * 4));
    CHECK(cudaMalloc(&ln, R * 4));
    CHECK(cudaMalloc(&runs, size_t(BLOCKS) * most * sizeof(Found)));
    CHECK(cudaMalloc(&counts, BLOCKS * 4));
    CHECK(cudaMalloc(&a.meta, BLOCKS * sizeof(TreeMeta)));
    CHECK(cudaMemcpy(qs, starts.data(), (R + 1) * 4, cudaMemcpyHostToDevice));
    CHECK(cudaMemcpy(ln, len.data(), R * 4, cudaMemcpyHostToDevice));
    a.q_start = qs;
    a.kv_len = ln;
    a.R = R;
    a.Tq = starts[R];
    a.Hk = 1;
    a.G = a.Hq = a.share = heads;
    a.max_len = (1 << 30);
    divide<<<BLOCKS, THREADS>>>(a, runs, most, counts);
    CHECK(cudaGetLastError());
    CHECK(cudaDeviceSynchronize());
    std::vector<Found> got(size_t(BLOCKS) * most);
    std::vector<int> count(BLOCKS);
    std::vector<TreeMeta> meta(BLOCKS);
    CHECK(cudaMemcpy(got.data(), runs, got.size() * sizeof(Found), cudaMemcpyDeviceToHost));
    CHECK(cudaMemcpy(count.data(), counts, BLOCKS * 4, cudaMemcpyDeviceToHost));
    CHECK(cudaMemcpy(meta.data(), a.meta, BLOCKS * sizeof(TreeMeta), cudaMemcpyDeviceToHost));
    for (void* p : {(void*)qs, (void*)ln, (void*)runs, (void*)counts, (void*)a.meta}) CHECK(cudaFree(p));

    int wrong = 0;
    int64_t busiest = 0, total = 0;
    std::vector<int> done(first[R], 0), from(first[R], -1), last(first[R], -1);  // tiles, first and last block of a group
    for (int b = 0; b < BLOCKS; ++b) {
        int64_t cost = 0;
        std::vector<int64_t> slots;
        for (int i = 0; i < count[b]; ++i) {
            const Found& x = got[size_t(b) * most + i];
            const int64_t g = first[x.r] + x.m;
            const int nt = tiles(x.r), light = nt - (leads ? masked(x.r) : 0);
            wrong += x.count < 1 || x.t0 != done[g] || x.t0 + x.count > nt;  // in order, block after block
            done[g] += x.count;
            wrong += last[g] != (from[g] < 0 ? -1 : b - 1);
            if (from[g] < 0) from[g] = b;
            last[g] = b;
            if (x.count == nt) wrong += x.slot != -1;
            else {
                wrong += x.slot != b * 2 + (x.t0 == 0 ? 1 : 0);
                slots.push_back(x.slot);
            }
            wrong += x.t0 > 0 && i > 0;
            cost += (leads ? kLead : 0) + x.count + kMasked * std::max(0, x.t0 + x.count - std::max(x.t0, light));
        }
        std::sort(slots.begin(), slots.end());
        wrong += std::unique(slots.begin(), slots.end()) != slots.end();
        busiest = std::max(busiest, cost);
        total += cost;
    }
    for (int r = 0; r < R; ++r)
        for (int64_t g = first[r]; g < first[r + 1]; ++g) wrong += done[g] != tiles(r);
    // what the join is told: the group that a block goes on with, and its first and last block
    for (int b = 0; b < BLOCKS; ++b) {
        const Found* x = count[b] ? &got[size_t(b) * most] : nullptr;
        if (!x || x->t0 == 0) {
            wrong += meta[b].nt != 0;
            continue;
        }
        const int64_t g = first[x->r] + x->m;
        wrong += meta[b].r != x->r || meta[b].m != x->m || meta[b].nt < 1;
        wrong += meta[b].u0 / meta[b].chunk != from[g] || (meta[b].u0 + meta[b].nt - 1) / meta[b].chunk != last[g];
    }
    const int64_t even = (total + BLOCKS - 1) / BLOCKS;
    printf("%s: %lld groups, busiest block %lld, mean %lld, %d wrong\n", what, (long long)first[R], (long long)busiest,
           (long long)even, wrong);
    return wrong != 0 || (leads && busiest > even + 2 * kLead + kMasked + 1);
}

int main() {
    int bad = 0;
    bad += check("4096 of 4096, 1 head", {4096}, {4096}, 1);
    bad += check("1024 of 5120, 4 heads", {1024}, {5120}, 4);
    bad += check("1024 of 8192, 16 heads", {1024}, {8192}, 16);
    bad += check("2048 of 2048, 16 heads", {2048}, {2048}, 16);
    bad += check("chunks, 64 heads", {200, 228, 256}, {1031, 2565, 4099}, 64);
    bad += check("more drafts than rows", {500, 70, 0, 900}, {100, 0, 7, 640}, 8);
    bad += check("one token", {1}, {131072}, 16);
    bad += check("nothing", {0, 0}, {5, 0}, 16);
    unsigned seed = 1;
    auto rnd = [&](int k) { return int((seed = seed * 1664525u + 1013904223u) >> 8) % k; };
    for (int i = 0; i < 60; ++i) {
        const int R = 1 + rnd(i % 3 ? 8 : 700), most = i % 3 ? 900 : 3;
        std::vector<int> n(R), len(R);
        for (int r = 0; r < R; ++r) n[r] = rnd(most + 1), len[r] = rnd(7) ? n[r] + rnd(i % 4 ? 3000 : 90) : rnd(200);
        char what[40];
        snprintf(what, sizeof what, "drawn %d", i);
        bad += check(what, n, len, 1 + rnd(130));
    }
    printf(bad ? "FAIL\n" : "ok\n");
    return bad != 0;
}
