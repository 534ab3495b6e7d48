// rope_tree_tile.cuh -- attention of more than 16 query rows a key head (trees
// of drafted tokens, chunks of prompts) over a paged cache, on tcgen05.
//
// Mathematics: that of rope_tree_narrow.cuh, on tiles of 128 query rows.  Two
// differences.  The maximum that weights refer to may lag: it moves (and O
// and l shrink) only when the row's maximum has passed it by more than 2^8,
// so p reaches 2^8 at most and the sums stay exact in fp32; O lives in tensor
// memory, where rescaling it costs a read and a write of the whole
// accumulator.  And the fp16 bias is 2^7, which leaves p below 2^15.
//
// What bounds it.  128 x TN x (Dk + Dv) multiply-adds a tile against TN (Dk +
// Dv) cache elements: 128 query rows take 1024 cycles of tensor pipe a tile
// of 128 x 128 + 128, and 16-bit rows 2800 cycles of this card's HBM share per
// SM.  So up to 128 rows it is bound by HBM (8-bit: 1400 cycles), and beyond
// that by the tensor pipe and the exponentials.
//
// How.  One block an SM, 16 warps with one role each:
//   0-3, 4-7  two softmax groups.  A thread owns a query row (a lane of tensor
//             memory): it reads its row of s, makes p, writes p back over s as
//             16-bit pairs, and keeps m and l.
//   8-11      loads.  16-bit rows go from global to shared memory by cp.async;
//             8-bit rows to a ring of each thread's own and from there, as
//             fp16, to the tile.  Both put 128-byte lines of 64 lanes in the
//             128-byte swizzle, the layout that the tensor pipe takes for keys
//             (lanes contiguous along the sum) and values (along the columns)
//             alike.  Gathered by page, so pages of any size do.
//   12        the one thread that issues tcgen05.mma: s = q k into tensor
//             memory, O += p v with p from tensor memory.
// Each softmax group has its own s (128 columns) and O (128 columns), all 512
// of tensor memory, and its own chain s -> p -> O; while one group is at its
// softmax the tensor pipe works for the other.  Up to 128 query rows (PAIR
// false) the groups take the run's tiles in turn and are joined when it ends;
// beyond that (PAIR) they are two row tiles against the same cache tile, which
// then is read once for 256 rows.
//   Every wait is bounded: a wait that gives up sets `dead`, later waits
// return at once, and the run's rows come out as NaN.
#pragma once
#include "rope_tree_common.cuh"

namespace rope {

template <int STORE_, int DK_, int DV_, bool PAIR_>
struct TileCfg {
    static constexpr int STORE = STORE_, DK = DK_, DV = DV_;
    static constexpr bool PAIR = PAIR_;
    static constexpr bool kWide = STORE == ROPE_CACHE_BF16 || STORE == ROPE_CACHE_FP16;  // 16-bit codes
    static constexpr bool BF16 = STORE == ROPE_CACHE_BF16;
    static constexpr int TN = (kWide && DK <= 128) || DK == 64 ? 128 : 64;  // cache rows of a tile
    static constexpr int ROWS = PAIR ? 256 : 128;
    static constexpr int QTILE = 128 * DK * 2, Q_BYTES = QTILE * (PAIR ? 2 : 1);
    static constexpr int K_BYTES = TN * DK * 2, TILE = K_BYTES + TN * DV * 2;
    // 8-bit: what the load warps hold as codes (and two scales a thread), and
    // the scales of a tile with the largest value's scale of each load warp
    static constexpr int RAW = kWide ? 0 : TN * (DK + DV) + 1024;
    static constexpr int RAWS = kWide ? 0 : (PAIR && DK == 192 ? 1 : 3);
    static constexpr int SC = kWide ? 0 : TN * 8 + 16;
    static constexpr int MISC = 3072;
    static constexpr int kSmemMax = 232448;
    static constexpr int FIT = (kSmemMax - MISC - Q_BYTES - RAW * RAWS) / (TILE + SC);
    static constexpr int STAGES = FIT > 4 ? 4 : FIT;
    static constexpr int TILES_AT = Q_BYTES;
    static constexpr int RAW_AT = TILES_AT + STAGES * TILE;
    static constexpr int SC_AT = RAW_AT + RAWS * RAW;
    static constexpr int MISC_AT = SC_AT + STAGES * SC;
    // in MISC: (m, l) of both groups, then TileSync
    static constexpr int ML_AT = MISC_AT, SYNC_AT = MISC_AT + 2048;
    static constexpr int SMEM = MISC_AT + MISC;
    static constexpr float kBias = BF16 ? 0.0f : 7.0f;
    static constexpr float kLag = 8.0f;
    static_assert(STAGES >= 2, "a tile in use and one on its way");
};

constexpr uint32_t kSpins = 1u << 20;  // tries of one wait before it gives up

struct TileSync {
    unsigned long long full[4], empty[4], s_full[2], p_full[2], o_full[2], q_full, done;
    uint32_t tmem;
    volatile uint32_t dead;
    volatile uint32_t patch[8];  // of run r at r % 8: values were taken out
};

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

__device__ __forceinline__ void bar_wait(unsigned long long* b, uint32_t parity, TileSync* s) {
    for (uint32_t i = 0; i < kSpins; ++i) {
        if (bar_test(b, parity)) return;
        if (s->dead) return;
    }
    s->dead = 1;
}

// The 256 threads of the softmax groups.
__device__ __forceinline__ void groups_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void to_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define ROPE_R8(r, i) "=f"(r[i]), "=f"(r[i + 1]), "=f"(r[i + 2]), "=f"(r[i + 3]), "=f"(r[i + 4]), "=f"(r[i + 5]), \
                      "=f"(r[i + 6]), "=f"(r[i + 7])
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

// Column of tensor memory of group w's s (and p) and O.
__host__ __device__ constexpr uint32_t s_col(int w) { return uint32_t(w) * 128; }
__host__ __device__ constexpr uint32_t o_col(int w) { return 256 + uint32_t(w) * 128; }

template <class C>
struct Tile {
    const TreeArgs& a;
    char* smem;
    TileSync* sync;
    uint32_t tmem;

    // ---------------------------------------------------------- loads

    // Rows of this warp: [rows0, rows0 + PER) of a tile; lane l looks up row
    // rows0 + l.  `at` is -1 for a row that is not there.
    struct Found {
        int64_t k, v;  // bytes from the cache's start, -1: none
        int64_t ks, vs;
    };
    static constexpr int PER = C::TN / 4;

    __device__ __forceinline__ Found find(const RunAt& x, int tile, int rows0, int lane) const {
        Found f{-1, -1, -1, -1};
        const int j = tile * C::TN + rows0 + lane;
        if (lane < PER && j < x.rq.len) {
            uint32_t p, off;
            a.div_page.divmod(uint32_t(j), p, off);
            const int page = __ldg(a.table + int64_t(x.r) * a.table_stride + p);
            if (page >= 0 && page < a.pages) {
                f.k = page * a.k_st[0] + int64_t(off) * a.k_st[1] + int64_t(x.h) * a.k_st[2];
                f.v = page * a.v_st[0] + int64_t(off) * a.v_st[1] + int64_t(x.h) * a.v_st[2];
                if constexpr (!C::kWide) {
                    f.ks = page * a.ks_st[0] + int64_t(off) * a.ks_st[1] + int64_t(x.h) * a.ks_st[2];
                    f.vs = page * a.vs_st[0] + int64_t(off) * a.vs_st[1] + int64_t(x.h) * a.vs_st[2];
                }
            }
        }
        return f;
    }

    // Where 16 bytes (8 lanes from 8 ch) of row `row` lie in a 16-bit tile.
    static __device__ __forceinline__ uint32_t line_at(int row, int ch) {
        return uint32_t(ch >> 3) * (C::TN * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
    }

    // One side (keys or values) of a 16-bit tile.
    template <int D>
    __device__ __forceinline__ void copy_side(const char* base, int64_t mine, uint32_t to, int rows0, int lane,
                                              int dim) const {
        constexpr int CH = D / 8;  // chunks of a row
#pragma unroll
        for (int i = 0; i < PER * CH / 32; ++i) {
            const int idx = lane + 32 * i, row = idx / CH, ch = idx % CH;
            const int64_t at = __shfl_sync(0xffffffffu, mine, row);
            const bool ok = at >= 0 && ch * 8 < dim;
            copy16(to + line_at(rows0 + row, ch), ok ? base + at + ch * 16 : base, ok);
        }
    }

    // The same for 8-bit codes: the thread's own 16 bytes of `raw` (chunk i of
    // thread t at 16 (128 i + t)).
    template <int D>
    __device__ __forceinline__ void copy_codes(const char* base, int64_t mine, uint32_t raw, int lane, int dim) const {
        constexpr int CH = D / 16;
#pragma unroll
        for (int i = 0; i < PER * CH / 32; ++i) {
            const int idx = lane + 32 * i, row = idx / CH, ch = idx % CH;
            const int64_t at = __shfl_sync(0xffffffffu, mine, row);
            const bool ok = at >= 0 && ch * 16 < dim;
            copy16(raw + i * 2048, ok ? base + at + ch * 16 : base, ok);
        }
    }

    template <int D>
    __device__ __forceinline__ void widen_codes(uint32_t raw, uint32_t to, int rows0, int lane) const {
        constexpr int CH = D / 16;
#pragma unroll
        for (int i = 0; i < PER * CH / 32; ++i) {
            const int idx = lane + 32 * i, row = rows0 + idx / CH, ch = idx % CH;
            uint32_t w[4], h[8];
            lds128(w, raw + i * 2048);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[2 * j] = codes_to_half2<C::STORE, false>(w[j]);
                h[2 * j + 1] = codes_to_half2<C::STORE, true>(w[j]);
            }
            sts128(to + line_at(row, 2 * ch), h[0], h[1], h[2], h[3]);
            sts128(to + line_at(row, 2 * ch + 1), h[4], h[5], h[6], h[7]);
        }
    }

    // 16-bit values of drafted rows that are not finite become zeros (see
    // add_not_finite); the thread looks at what it copied itself.
    static __device__ __noinline__ void take_out_not_finite(TileSync* sync, uint32_t to, int rows0, int lane,
                                                            int from, uint32_t run) {
        constexpr int CH = C::DV / 8;
        for (int i = 0; i < PER * CH / 32; ++i) {
            const int idx = lane + 32 * i, row = rows0 + idx / CH, ch = idx % CH;
            if (row < from) continue;
            uint32_t w[4];
            lds128(w, to + line_at(row, ch));
            bool found = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool lo = not_finite<C::STORE>(w[j] & 0xffffu), hi = not_finite<C::STORE>(w[j] >> 16);
                if (lo || hi) {
                    found = true;
                    w[j] = (lo ? 0u : w[j] & 0xffffu) | (hi ? 0u : w[j] & 0xffff0000u);
                }
            }
            if (found) {
                sts128(to + line_at(row, ch), w[0], w[1], w[2], w[3]);
                sync->patch[run] = 1;
            }
        }
    }

    static __device__ __forceinline__ void wait_all_but(uint32_t newer) {
        if (newer == 0) copies_wait<0>();
        else if (newer == 1) copies_wait<1>();
        else if (newer == 2) copies_wait<2>();
        else copies_wait<3>();
    }

    // The load warps.  Tiles are issued as far ahead as the ring allows, across
    // runs, and arrive in order: a thread's copies are complete, its fence lets
    // the tensor pipe see them, its arrival is one of 128.
    __device__ __forceinline__ void loads(const Place& place) const {
        const int lane = int(threadIdx.x) & 31, warp = (int(threadIdx.x) >> 5) & 3;
        const int rows0 = warp * PER;
        constexpr uint32_t AHEAD = C::kWide ? C::STAGES : C::RAWS;
        Walk<C::ROWS, C::TN> walk(a, place);
        RunAt x;
        bool more = walk.next(x);
        uint32_t run = 0, issued = 0, arrived = 0;
        int it = 0;
        // of each tile on its way: the first row that is a drafted token's own
        // (8 bits) and its run modulo 8
        unsigned long long fifo = 0;
        Found next{-1, -1, -1, -1};
        if (more) next = find(x, x.t0, rows0, lane);

        while (true) {
            while (more && issued - arrived < AHEAD) {
                if (C::kWide && issued >= uint32_t(C::STAGES)) {
                    // the tile's place must be free; while others are on their
                    // way, they come first
                    const uint32_t st = issued % C::STAGES, par = (issued / C::STAGES - 1) & 1;
                    if (issued == arrived) bar_wait(&sync->empty[st], par, sync);
                    else if (!__all_sync(0xffffffffu, bar_test(&sync->empty[st], par) || sync->dead)) break;
                }
                if constexpr (C::kWide) {
                    const uint32_t to = smem_addr(smem + C::TILES_AT + issued % C::STAGES * C::TILE);
                    copy_side<C::DK>(a.k, next.k, to, rows0, lane, a.Dk);
                    copy_side<C::DV>(a.v, next.v, to + C::K_BYTES, rows0, lane, a.Dv);
                    const int from = x.rq.len - x.rq.n - (x.t0 + it) * C::TN;
                    fifo |= (unsigned long long)(min(max(from, 0), 255) | (run & 7) << 8) << (16 * (issued - arrived));
                } else {
                    const uint32_t raw = smem_addr(smem + C::RAW_AT + issued % AHEAD * C::RAW);
                    const uint32_t mine = raw + (int(threadIdx.x) & 127) * 16;
                    copy_codes<C::DK>(a.k, next.k, mine, lane, a.Dk);
                    copy_codes<C::DV>(a.v, next.v, mine + C::TN * C::DK, lane, a.Dv);
                    if (lane < PER) {
                        const uint32_t sc = raw + C::TN * (C::DK + C::DV) + (int(threadIdx.x) & 127) * 8;
                        copy4(sc, next.ks >= 0 ? a.ks + next.ks : a.ks, next.ks >= 0);
                        copy4(sc + 4, next.vs >= 0 ? a.vs + next.vs : a.vs, next.vs >= 0);
                    }
                }
                copies_commit();
                ++issued;
                if (++it == x.count) {
                    more = walk.next(x);
                    ++run;
                    it = 0;
                }
                if (more) next = find(x, x.t0 + it, rows0, lane);
            }
            if (issued == arrived) break;
            wait_all_but(issued - arrived - 1);
            const uint32_t st = arrived % C::STAGES;
            const uint32_t to = smem_addr(smem + C::TILES_AT + st * C::TILE);
            if constexpr (C::kWide) {
                const int from = int(fifo & 255);
                if (from < C::TN) 
                    take_out_not_finite(sync, to + C::K_BYTES, rows0, lane, from, uint32_t(fifo >> 8) & 7);
                fifo >>= 16;
            } else {
                if (arrived >= uint32_t(C::STAGES))
                    bar_wait(&sync->empty[st], (arrived / C::STAGES - 1) & 1, sync);
                const uint32_t raw = smem_addr(smem + C::RAW_AT + arrived % AHEAD * C::RAW);
                const uint32_t mine = raw + (int(threadIdx.x) & 127) * 16;
                widen_codes<C::DK>(mine, to, rows0, lane);
                widen_codes<C::DV>(mine + C::TN * C::DK, to + C::K_BYTES, rows0, lane);
                float* sc = reinterpret_cast<float*>(smem + C::SC_AT + st * C::SC);
                float v = 0.0f;
                if (lane < PER) {
                    const float2 y = *reinterpret_cast<const float2*>(
                        smem + C::RAW_AT + arrived % AHEAD * C::RAW + C::TN * (C::DK + C::DV) +
                        (int(threadIdx.x) & 127) * 8);
                    sc[rows0 + lane] = y.x;
                    sc[C::TN + rows0 + lane] = y.y;
                    v = y.y;
                }
#pragma unroll
                for (int d = 16; d; d /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                if (lane == 0) sc[2 * C::TN + warp] = v;
            }
            to_async_proxy();
            bar_arrive(&sync->full[st]);
            ++arrived;
        }
    }

    // ---------------------------------------------------------- products

    // The thread that issues the products.  A group's chain is s, (its
    // softmax), O; whichever group's next step is ready goes next.
    __device__ __forceinline__ void products(const Place& place) const {
        constexpr uint32_t QK = mma_shape<C::BF16, C::TN, false>();
        constexpr uint32_t PV = mma_shape<C::BF16, C::DV, true>();
        Walk<C::ROWS, C::TN> walk(a, place);
        RunAt x;
        uint32_t before = 0, q_par = 0, p_par[2] = {0, 0};
        const uint32_t q_at = smem_addr(smem), tiles = smem_addr(smem + C::TILES_AT);
        while (walk.next(x)) {
            bar_wait(&sync->q_full, q_par, sync);
            q_par ^= 1;
            tmem_after();
            const int nv = C::PAIR ? 2 * x.count : x.count;  // steps; step v is group v & 1's
            int s_next[2] = {0, 1}, p_next[2] = {0, 1}, left = nv;
            uint32_t spins = 0;
            while (left > 0) {
                bool moved = false;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (s_next[w] > p_next[w] && bar_test(&sync->p_full[w], p_par[w])) {
                        tmem_after();
                        const int v = p_next[w], t = C::PAIR ? v >> 1 : v;
                        const uint32_t st = (before + t) % C::STAGES;
                        const uint32_t vs = tiles + st * C::TILE + C::K_BYTES;
#pragma unroll
                        for (int k = 0; k < C::TN / 16; ++k)
                            mma_ts(tmem + o_col(w), tmem + s_col(w) + 8 * k, smem_matrix(vs + k * 2048, C::TN * 128),
                                   PV, v > 1 || k > 0);
                        p_par[w] ^= 1;
                        p_next[w] += 2;
                        if (!C::PAIR || (p_next[1 - w] >> 1) > t) mma_commit(&sync->empty[st]);
                        if (p_next[w] >= nv) mma_commit(&sync->o_full[w]);
                        --left;
                        moved = true;
                    }
                    if (s_next[w] == p_next[w] && s_next[w] < nv) {
                        const int t = C::PAIR ? s_next[w] >> 1 : s_next[w];
                        const uint32_t n = before + t, st = n % C::STAGES;
                        if (bar_test(&sync->full[st], (n / C::STAGES) & 1)) {
                            tmem_after();
                            const uint32_t ks = tiles + st * C::TILE, q = q_at + (C::PAIR ? w * C::QTILE : 0);
#pragma unroll
                            for (int k = 0; k < C::DK / 16; ++k)
                                mma_ss(tmem + s_col(w), smem_matrix(q + (k >> 2) * 16384 + (k & 3) * 32, 16),
                                       smem_matrix(ks + (k >> 2) * (C::TN * 128) + (k & 3) * 32, 16), QK, k > 0);
                            mma_commit(&sync->s_full[w]);
                            s_next[w] += 2;
                            moved = true;
                        }
                    }
                }
                if (moved) spins = 0;
                else if (sync->dead || ++spins > kSpins) {
                    sync->dead = 1;
                    break;
                }
            }
            before += x.count;
        }
        mma_commit(&sync->done);
        for (uint32_t i = 0; i < kSpins && !bar_test(&sync->done, 0); ++i) {
        }
    }

    // ---------------------------------------------------------- softmax

    // The row tile's queries: 16-bit as they are, or fp16 in [-2, 2); returns
    // what the row's s is multiplied by.
    __device__ __forceinline__ float stage_queries(const RunAt& x, int w, int row) const {
        const int at = x.m * C::ROWS + (C::PAIR ? 128 * w : 0) + row;
        const bool there = at < x.rq.n * a.G;
        uint32_t tok = 0, g = 0;
        if (there) a.div_group.divmod(uint32_t(at), tok, g);
        const uint4* src = reinterpret_cast<const uint4*>(a.q + int64_t(x.rq.qs + int(tok)) * a.q_st[0] +
                                                          int64_t(x.h * a.G + int(g)) * a.q_st[1]);
        const int chunks = there ? a.Dk / 8 : 0;
        float factor = a.scale_log2, down = 1.0f;
        if constexpr (!C::kWide) {
            uint32_t most = 0;
#pragma unroll 4
            for (int ch = 0; ch < chunks; ++ch) {
                float f[8];
                widen8(__ldg(src + ch), a.bf16, f);
                most = max(most, most_of(f));
            }
            const float p = row_power(most);
            down = one_over_power(p);
            factor *= p;
        }
        // up to 128 rows, both groups' threads of a row take half of it each
        constexpr int CH = C::DK / 8, N = C::PAIR ? CH : CH / 2;
        const int first = C::PAIR ? 0 : w * N;
        const uint32_t to = smem_addr(smem) + (C::PAIR ? w * C::QTILE : 0) + row * 128;
#pragma unroll 4
        for (int i = 0; i < N; ++i) {
            const int ch = first + i;
            uint4 y = ch < chunks ? __ldg(src + ch) : make_uint4(0, 0, 0, 0);
            if constexpr (!C::kWide) {
                float f[8];
                widen8(y, a.bf16, f);
                y = half8(f, down);
            }
            sts128(to + (ch >> 3) * 16384 + (((ch & 7) ^ (row & 7)) << 4), y.x, y.y, y.z, y.w);
        }
        return factor;
    }

    // Four sums or maxima side by side.
    template <int N>
    static __device__ __forceinline__ float max_of(const float* s) {
        float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int j = 4; j < N; ++j) m[j & 3] = fmaxf(m[j & 3], s[j]);
        return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    }

    __device__ __forceinline__ void softmax(const Place& place, int w) const {
        const int tid = int(threadIdx.x), row = tid & 127;
        const uint32_t lanes = tmem + (uint32_t(row & 96) << 16);  // this warp's lanes
        float2* ml = reinterpret_cast<float2*>(smem + C::ML_AT);
        Walk<C::ROWS, C::TN> walk(a, place);
        RunAt x;
        uint32_t before = 0, run = 0, s_par = 0, o_par = 0;
        TreeMeta meta{0, place.chunk, 0, 0, 0, 0};
        while (walk.next(x)) {
            if (run == 0) meta = meta_of(place, x);
            const float factor = stage_queries(x, w, row);
            to_async_proxy();
            bar_arrive(&sync->q_full);

            const int rows = x.rq.n * a.G;
            const int at = x.m * C::ROWS + (C::PAIR ? 128 * w : 0) + row;
            const bool active = at - (row & 31) < rows;  // the warp has a row
            const int tok = min(int(a.div_group.div(uint32_t(at))), x.rq.n - 1);
            const int prefix = x.rq.len - x.rq.n, nv = C::PAIR ? 2 * x.count : x.count;
            float m = -INFINITY, l = 0.0f, vref = kLeastPower;

#pragma unroll 1
            for (int v = w; v < nv; v += 2) {
                const int t = C::PAIR ? v >> 1 : v, j0 = (x.t0 + t) * C::TN;
                const uint32_t n = before + t, st = n % C::STAGES;
                const float* sc = reinterpret_cast<const float*>(smem + C::SC_AT + st * C::SC);
                bar_wait(&sync->s_full[w], s_par, sync);
                s_par ^= 1;
                tmem_after();
                if (active) {
                    float s[C::TN];
#pragma unroll
                    for (int c = 0; c < C::TN; c += 32) tmem_ld32(s + c, lanes + s_col(w) + c);
                    tmem_wait_ld();
                    if constexpr (!C::kWide) {
                        bar_wait(&sync->full[st], (n / C::STAGES) & 1, sync);  // long since: the scales
#pragma unroll
                        for (int j = 0; j < C::TN; j += 4) {
                            const float4 y = *reinterpret_cast<const float4*>(sc + j);
                            s[j] *= y.x;
                            s[j + 1] *= y.y;
                            s[j + 2] *= y.z;
                            s[j + 3] *= y.w;
                        }
                    }
                    if (j0 + C::TN > prefix) {
#pragma unroll
                        for (int c = 0; c < C::TN; c += 32) {
                            const uint32_t bits = sees32(a, x.rq.qs, tok, prefix, x.rq.len, j0 + c);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!(bits >> j & 1u)) s[c + j] = -INFINITY;
                        }
                    }
                    const float top = max_of<C::TN>(s) * factor;
                    const bool up = top > m + C::kLag || (m == -INFINITY && top > m);
                    float shrink = 1.0f;
                    if (up) {
                        shrink = pow2(m - top);
                        m = top;
                        l *= shrink;
                    }
                    if constexpr (!C::kWide) {
                        const float4 y = *reinterpret_cast<const float4*>(sc + 2 * C::TN);
                        const float u = fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w));
                        if (u > vref) {
                            const float p = power_above(u);
                            shrink *= vref / p;
                            vref = p;
                        }
                    }
                    if (v > 1 && __any_sync(0xffffffffu, shrink != 1.0f)) {
#pragma unroll 1
                        for (int c = 0; c < C::DV; c += 32) {
                            float o[32];
                            tmem_ld32(o, lanes + o_col(w) + c);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] *= shrink;
                            tmem_st32(lanes + o_col(w) + c, reinterpret_cast<const uint32_t*>(o));
                        }
                    }
                    const float base = C::kBias - (m == -INFINITY ? 0.0f : m);
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    const float back = C::kWide ? 1.0f : one_over_power(vref);
#pragma unroll
                    for (int c = 0; c < C::TN; c += 32) {
                        uint32_t p[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            float4 u = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                            if constexpr (!C::kWide) u = *reinterpret_cast<const float4*>(sc + C::TN + c + j);
                            float e[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                e[i] = pow2(fmaf(s[c + j + i], factor, base));
                                sum[i] += e[i];
                            }
                            if constexpr (!C::kWide) {
                                // a row that is not seen adds nothing, whatever its scale
                                e[0] = e[0] == 0.0f ? 0.0f : e[0] * (u.x * back);
                                e[1] = e[1] == 0.0f ? 0.0f : e[1] * (u.y * back);
                                e[2] = e[2] == 0.0f ? 0.0f : e[2] * (u.z * back);
                                e[3] = e[3] == 0.0f ? 0.0f : e[3] * (u.w * back);
                            }
                            p[j / 2] = pack2<C::BF16>(e[0], e[1]);
                            p[j / 2 + 1] = pack2<C::BF16>(e[2], e[3]);
                        }
                        tmem_st16(lanes + s_col(w) + c / 2, p);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_wait_st();
                }
                tmem_before();
                bar_arrive(&sync->p_full[w]);
            }
            if (w < nv) {
                bar_wait(&sync->o_full[w], o_par, sync);
                o_par ^= 1;
                tmem_after();
            }
            finish(x, w, row, at, at < rows, active, nv, m, l, vref, sync->patch[run & 7] != 0, ml, lanes);
            tmem_before();
            groups_sync();  // queries, O and ml are done with
            if (tid == 0) sync->patch[run & 7] = 0;
            before += x.count;
            ++run;
        }
        if (tid == 0) a.meta[blockIdx.x] = meta;
    }

    // The results of a run.
    __device__ __forceinline__ void finish(const RunAt& x, int w, int row, int at, bool there, bool active, int nv,
                                           float m, float l, float vref, bool patch, float2* ml,
                                           uint32_t lanes) const {
        float f = C::kWide ? 1.0f : vref;
        if (C::PAIR || nv == 1) {
            // one group has the row to itself
            if ((C::PAIR || w == 0) && active) {
#pragma unroll 1
                for (int c = 0; c < C::DV; c += 32) {
                    float o[32];
                    tmem_ld32(o, lanes + o_col(w) + c);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] *= f;
                    if (there) put(x, (C::PAIR ? 128 * w : 0) + row, at, c, o, m, l, patch);
                }
            }
            return;
        }
        // the groups took turns at the tiles: group 1's sums go through shared
        // memory (the queries' place, a column of rows at a time) to group 0
        ml[w * 128 + row] = make_float2(m, l);
        groups_sync();
        const float2 other = ml[(1 - w) * 128 + row];
        const float top = fmaxf(m, other.x), base = top == -INFINITY ? 0.0f : top;
        const float own = pow2(m - base);
        f *= own;
        l = l * own + other.y * pow2(other.x - base);
        float* give = reinterpret_cast<float*>(smem);
#pragma unroll 1
        for (int c = 0; c < C::DV; c += 32) {
            float o[32];
            if (active) {
                tmem_ld32(o, lanes + o_col(w) + c);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] *= f;
                if (w == 1) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) give[j * 128 + row] = o[j];
                }
            }
            groups_sync();
            if (active && w == 0) {
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] += give[j * 128 + row];
                if (there) put(x, row, at, c, o, top, l, patch);
            }
            groups_sync();
        }
    }

    // 32 columns from c of one row: the result, or the part.
    __device__ __forceinline__ void put(const RunAt& x, int row, int at, int c, float* o, float top, float l,
                                        bool patch) const {
        if constexpr (C::kWide) {
            if (patch) add_not_finite<C::STORE, C::TN, 32>(a, x, at, c, o);
        }
        if (sync->dead) l = NAN;
        if (x.slot >= 0) {
            float4* to = reinterpret_cast<float4*>(a.part + (x.slot * C::ROWS + row) * C::DV + c);
#pragma unroll
            for (int j = 0; j < 8; ++j) to[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            if (c == 0) a.part_ml[x.slot * C::ROWS + row] = make_float2(top, l);
            return;
        }
        const OutAt to = out_at(a, x.rq.qs, x.h, at);
        if (c == 0 && to.lse) *to.lse = lse_of(top, l, C::kBias);
        const float f = l == 0.0f ? 0.0f : 1.0f / l;  // a token that has seen no row gives zeros
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            if (c + j >= a.Dv) break;
            uint4 y;
            if (a.bf16)
                y = make_uint4(pack2<true>(o[j] * f, o[j + 1] * f), pack2<true>(o[j + 2] * f, o[j + 3] * f),
                               pack2<true>(o[j + 4] * f, o[j + 5] * f), pack2<true>(o[j + 6] * f, o[j + 7] * f));
            else
                y = make_uint4(pack2<false>(o[j] * f, o[j + 1] * f), pack2<false>(o[j + 2] * f, o[j + 3] * f),
                               pack2<false>(o[j + 4] * f, o[j + 5] * f), pack2<false>(o[j + 6] * f, o[j + 7] * f));
            *reinterpret_cast<uint4*>(to.out + (c + j) * 2) = y;
        }
    }
};

template <class C>
__global__ void __launch_bounds__(kTileThreads, 1) rope_tree_tile_kernel(const __grid_constant__ TreeArgs a) {
    extern __shared__ __align__(1024) char smem[];
    TileSync* sync = reinterpret_cast<TileSync*>(smem + C::SYNC_AT);
    const int warp = int(threadIdx.x) >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            bar_init(&sync->full[i], 128);
            bar_init(&sync->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sync->s_full[i], 1);
            bar_init(&sync->p_full[i], 128);
            bar_init(&sync->o_full[i], 1);
        }
        bar_init(&sync->q_full, 256);
        bar_init(&sync->done, 1);
        sync->dead = 0;
        for (int i = 0; i < 8; ++i) sync->patch[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sync->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    after_predecessor();
    const Place place = find_place<C::ROWS, C::TN, kTileThreads>(a, reinterpret_cast<int64_t*>(smem + C::ML_AT));
    tmem_before();
    __syncthreads();
    tmem_after();
    const Tile<C> tile{a, smem, sync, sync->tmem};

    // registers: 128 a thread at launch; 256 x 192 + 128 x 80 + 128 x 48 of
    // the same 65536
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        tile.softmax(place, warp >> 2);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        tile.loads(place);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (threadIdx.x == 12 * 32) tile.products(place);
        __syncwarp();
    }
    tmem_before();
    __syncthreads();
    if (warp == 12) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sync->tmem));
    }
}

template <int STORE, int DK, int DV, bool PAIR>
TreeKernel tile_kernel() {
    using C = TileCfg<STORE, DK, DV, PAIR>;
    return TreeKernel{reinterpret_cast<const void*>(&rope_tree_tile_kernel<C>),
                      reinterpret_cast<const void*>(&rope_tree_join_kernel<C::ROWS, DV>), C::SMEM, kTileThreads,
                      C::kBias};
}

}  // namespace rope
