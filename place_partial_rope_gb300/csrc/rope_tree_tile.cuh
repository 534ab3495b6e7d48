// rope_tree_tile.cuh -- attention of many query rows a key head (batches of tokens,
// trees of drafted tokens, chunks of prompts) over a paged cache, on tcgen05.
//
// Mathematics: that of rope_tree_narrow.cuh, on tiles of 128 query rows.  Two
// differences.  The maximum that weights refer to may lag: it moves (and O
// and l shrink) only when the row's maximum has passed it by more than 2^8,
// so p reaches 2^8 at most and the sums stay exact in fp32; O lives in tensor
// memory, where rescaling it costs a read and a write of the whole
// accumulator.  And the fp16 bias is 2^7, which leaves p below 2^15.  8-bit: O
// and l are both kept in units of 1 / w (w the power of two above the scales of the
// values that the query row sees), so that a weight is 2^(s - m - log2 w) u, one
// product; w starts at 2^-80.
//
// What bounds it.  128 x TN x (Dk + Dv) multiply-adds a tile against TN (Dk +
// Dv) cache elements: 128 query rows take 1024 cycles of tensor pipe a tile
// of 128 x 128 + 128, and 16-bit rows 2800 cycles of this card's HBM share per
// SM.  So up to 128 rows 16 bits are bound by HBM (32 requests of 8000 rows, 8
// key heads: 182 us, 5.8 TB/s), and a pair of tiles by the chain s -> p -> O of
// its two groups: 12 requests of 6000 to 8200 rows and 240 to 256 query rows,
// 103 us, 0.43 of the measured matrix rate, the tensor pipe 40 % busy.  (The
// product on the first half of a row's weights, while the thread was at the second,
// took 121 us, not 105.)  8-bit rows would take 1400 cycles of HBM and take 3000: each
// code passes through shared memory four times and the helpers' and groups' code
// presses on the instruction cache (86 % of its requests hit): 48 requests of 90 to
// 12000 rows, 223 us, 2.8 TB/s.  (24 warps, twice the helpers: no faster.)
//
// How.  One block an SM, 16 warps with one role each:
//   0-3, 4-7  two softmax groups.  A thread owns a query row (a lane of tensor
//             memory): it reads its row of s, makes p, writes p back over s as
//             16-bit pairs, and keeps m and l.
//   13        fetches tiles by tensor copies, boxes of rows of one page, keys
//             and values in rings of their own.
//   8-11, 14, 15  helpers.  16-bit rows land in the layout that the tensor
//             pipe takes (lines of 64 lanes in the 128-byte swizzle; the same
//             for keys, whose lanes run along the sum, and values, whose lanes
//             run along the columns), and helpers touch only the last tiles of a
//             request.  8-bit rows land as codes, and helpers write them to
//             such tiles as fp16, one team of 96 threads keys and one values.
//   12        the one thread that issues tcgen05.mma: s = q k into tensor
//             memory, O += p v with p from tensor memory.
// Each softmax group has its own s (128 columns) and O (128 columns), all 512
// of tensor memory, and its own chain s -> p -> O; while one group is at its
// softmax the tensor pipe works for the other.  Up to 128 query rows (PAIR
// false) the groups take the run's tiles in turn and are joined when it ends;
// beyond that (PAIR) they are two row tiles against the same cache tile, which
// then is read once for 256 rows.
//   Tiles of up to 64 query rows (ROWS 64) are in tensor memory twice, as the upper
// and the lower 64 lanes, and each copy sees to half the columns: its weights in
// the other half are zeros, so the two O's are parts that add up.  So all 256
// threads of the groups have work.
//   The fetching warp alone walks the division of the work (request, head, tiles);
// it writes each run down in shared memory for the others.
//   Every wait is bounded, to some seconds: one that gives up sets `dead`, later
// waits return at once, the threads of a role leave together, fetches under way
// are waited for, and every result that the block has a share in becomes NaN.
//   Page sizes that are no multiple of 8 are left to rope_tree_narrow.cuh.
#pragma once
#include <cuda.h>

#include "rope_tree_common.cuh"

namespace rope {

template <int STORE_, int DK_, int DV_, int ROWS_>
struct TileCfg {
    static constexpr int STORE = STORE_, DK = DK_, DV = DV_;
    static constexpr int ROWS = ROWS_;  // query rows of a tile: 64, 128 or 256
    static constexpr bool PAIR = ROWS == 256;
    static constexpr int SPLIT = PAIR ? 1 : 128 / ROWS;  // copies of the rows in tensor memory
    static constexpr bool kWide = STORE == ROPE_CACHE_BF16 || STORE == ROPE_CACHE_FP16;  // 16-bit codes
    static constexpr bool BF16 = STORE == ROPE_CACHE_BF16;
    // cache rows of a tile: 128 where shared memory holds two tiles of that
    // (a product of 64 columns takes three quarters of the time of 128)
    static constexpr int TN = DK == 64 || (!PAIR && (kWide || DK == 128)) || (kWide && DK == 128) ? 128 : 64;
    static constexpr int COLS = TN / SPLIT;  // columns of s that a thread sees to
    static constexpr int QTILE = 128 * DK * 2, Q_BYTES = QTILE * (PAIR ? 2 : 1);
    // keys and values have rings of their own: a tile's keys are done with when
    // s is there, its values only after the softmax
    static constexpr int K_SLOT = TN * DK * 2, V_SLOT = TN * DV * 2;
    // 8-bit: the codes of a tile's keys or values, before they become fp16
    static constexpr int RAW = kWide ? 0 : TN * DK;
    static constexpr int RAWS = kWide ? 0 : TN == 128 && DK == 128 ? 3 : 4;
    static constexpr int ML = PAIR ? 0 : 2048, FACTORS = kWide ? 0 : ROWS * 4, MISC = ML + FACTORS + 1024;
    static constexpr int kSmemMax = 232448;
    static constexpr int fit(int slots) {
        return Q_BYTES + slots * (K_SLOT + V_SLOT) + RAWS * RAW + (kWide ? 0 : (slots + 2) * (TN * 8 + 16)) + MISC <=
               kSmemMax;
    }
    static constexpr int SLOTS = fit(4) ? 4 : fit(3) ? 3 : 2;
    // scales: a tile's outlive its keys' slot until the softmax, at most two
    // tiles on
    static constexpr int SCS = SLOTS + 2, SC = kWide ? 0 : TN * 8 + 16;
    static constexpr int K_AT = Q_BYTES, V_AT = K_AT + SLOTS * K_SLOT;
    static constexpr int RAW_AT = V_AT + SLOTS * V_SLOT;
    static constexpr int SC_AT = RAW_AT + RAWS * RAW;
    static constexpr int MISC_AT = SC_AT + SCS * SC;
    // in MISC: (m, l) of a row's sources, the rows' factors, TileSync
    static constexpr int ML_AT = MISC_AT, FACTOR_AT = ML_AT + ML, SYNC_AT = FACTOR_AT + FACTORS;
    static constexpr int SMEM = MISC_AT + MISC;
    static constexpr float kBias = BF16 ? 0.0f : 7.0f;
    static constexpr float kLag = 8.0f;
    static constexpr int kSyncMax = 896;
    static_assert(SYNC_AT + kSyncMax <= SMEM, "TileSync");
    static_assert(fit(SLOTS), "two tiles fit");
};

constexpr uint32_t kSpins = 1u << 20;  // tries of one wait before it gives up: 1.5 s and more
constexpr uint32_t kPolls = 1u << 26;  // looks of a thread that does not pause

struct TileSync {
    unsigned long long k_full[4], k_empty[4], v_full[4], v_empty[4];
    unsigned long long fix_full[4];                // 16-bit: values that the helpers see to first
    unsigned long long raw_full[4], raw_empty[4];  // 8-bit: codes
    unsigned long long s_full[2], p_full[2], o_full[2], q_full, done;
    uint32_t tmem;
    volatile uint32_t dead;
    volatile uint32_t patch[8];  // of run r at r % 8: values were taken out
    volatile uint32_t runs;      // runs that are in `run`, and
    volatile uint32_t last;      // how many there will be (~0: not known yet)
    volatile uint32_t beat;      // 16-bit: tiles fetched
    RunAt run[8];                // run r at r % 8: the fetching warp, which is ahead, writes them for the others
};
static_assert(sizeof(TileSync) <= TileCfg<ROPE_CACHE_FP8, 64, 64, 64>::kSyncMax, "its place in shared memory");

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

__device__ __forceinline__ void bar_wait(unsigned long long* b, uint32_t parity, TileSync* s) {
    for (uint32_t i = 0; i < kSpins; ++i) {
        if (bar_test(b, parity)) return;
        if (s->dead) return;
    }
    s->dead = 1;
}

// For those that may rightly wait for the whole of a run (16-bit helpers, whose
// tiles are its last; 7 s for 2^29 rows and 256 query rows): gives up when no
// tile has been fetched between two such stretches.
__device__ __forceinline__ void bar_wait_run(unsigned long long* b, uint32_t parity, TileSync* s) {
    for (uint32_t seen = ~0u;;) {
        for (uint32_t i = 0; i < kSpins; ++i) {
            if (bar_test(b, parity)) return;
            if (s->dead) return;
        }
        const uint32_t now = s->beat;
        if (now == seen) break;
        seen = now;
    }
    s->dead = 1;
}

// The 256 threads of the softmax groups.
__device__ __forceinline__ void groups_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The 192 threads that see to tiles between the fetch and the products; 8-bit:
// one half of them to keys, one to values.
constexpr int kHelpers = 192, kTeam = 96;
__device__ __forceinline__ void helpers_sync() { asm volatile("bar.sync 2, 192;" ::: "memory"); }

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

// Two fp32 operations in one instruction, each rounded as the single one.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long x, y, z, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    memcpy(&z, &c, 8);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    float2 r;
    memcpy(&r, &d, 8);
    return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long x, y, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    float2 r;
    memcpy(&r, &d, 8);
    return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long x, y, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    float2 r;
    memcpy(&r, &d, 8);
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Column of tensor memory of group w's s (and p) and O.
__host__ __device__ constexpr uint32_t s_col(int w) { return uint32_t(w) * 128; }
__host__ __device__ constexpr uint32_t o_col(int w) { return 256 + uint32_t(w) * 128; }

template <class C>
struct Tile {
    using Cfg = C;
    const TreeArgs& a;
    char* smem;
    TileSync* sync;
    uint32_t tmem;

    // ---------------------------------------------------------- loads

    // A tile's cache rows lie in boxes of a.box rows of one page (a power of
    // two, 8 or more).  A lane asks for its box's page a tile ahead.
    struct Look {
        int page;  // as the table says; -1: no such rows
        uint32_t off;
    };

    __device__ __forceinline__ Look look(const RunAt& x, int j) const {
        Look f{-1, 0};
        if (j < x.rq.len) {
            uint32_t p;
            a.div_page.divmod(uint32_t(j), p, f.off);
            f.page = __ldg(a.table + int64_t(x.r) * a.table_stride + p);
        }
        return f;
    }

    // The keys or values of a tile (16-bit: 64 lanes of a row to a line, in
    // planes; 8-bit: rows of codes) into shared memory.
    __device__ __forceinline__ void fetch(const CUtensorMap* map, int dim, const Look& f, int h, uint32_t to, int lane,
                                          unsigned long long* bar) const {
        if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)),
                         "r"(C::TN * dim * (C::kWide ? 2 : 1))
                         : "memory");
        __syncwarp();
        if (lane < C::TN / a.box) {
            const int line = C::kWide ? 128 : dim;
#pragma unroll 1
            for (int p = 0; p < (C::kWide ? dim : 64); p += 64)
                asm volatile(
                    "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                    "[%1, {%2, %3, %4, %5}], [%6];" ::"r"(to + p * (C::TN * 2) + lane * a.box * line),
                    "l"(map), "r"(p), "r"(h), "r"(int(f.off)), "r"(f.page), "r"(smem_addr(bar))
                    : "memory");
        }
    }

    // The fetching warp writes run r down for the other roles.  It is at most a
    // few tiles ahead of them (the rings' places), so eight places do.
    __device__ __forceinline__ void publish(const RunAt& x, uint32_t r, bool there, int lane) const {
        if (lane == 0) {
            if (there) {
                sync->run[r & 7] = x;
                __threadfence_block();
                sync->runs = r + 1;
            } else {
                __threadfence_block();
                sync->last = r;
            }
        }
        __syncwarp();
    }

    // Run r, when the block has one.  IDLE: of a role that may wait for a whole run
    // (see bar_wait_run).
    template <bool IDLE = false>
    __device__ __forceinline__ bool take(uint32_t r, RunAt& x) const {
        for (uint32_t seen = ~0u;;) {
            for (uint32_t i = 0; i < kPolls; ++i) {
                if (sync->runs > r) {
                    __threadfence_block();
                    x = sync->run[r & 7];
                    return true;
                }
                if (sync->last <= r || sync->dead) return false;
            }
            const uint32_t now = sync->beat;
            if (!IDLE || now == seen) break;
            seen = now;
        }
        sync->dead = 1;
        return false;
    }

    // The same for the N threads of a role that barrier ID counts, or (0) for the
    // lanes of a warp: all of them go on or none does.  Where a wait gives up just
    // as a run is written down, one thread may find the run and the next one
    // `dead`; a barrier that some do not reach would be waited for without end.
    template <int ID, int N = 32, bool IDLE = false>
    __device__ __forceinline__ bool take_all(uint32_t r, RunAt& x) const {
        const bool mine = take<IDLE>(r, x);
        if constexpr (ID == 0) return __all_sync(0xffffffffu, mine);
        __syncwarp();
        uint32_t all;
        asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.and.pred q, %2, %3, p;\n"
                     "selp.u32 %0, 1, 0, q;\n}"
                     : "=r"(all)
                     : "r"(uint32_t(mine)), "n"(ID), "n"(N)
                     : "memory");
        return all != 0;
    }

    // The warp that fetches tiles, keys and values in turn, across runs, as far
    // ahead as the rings allow.  A fetch that a wait before it did not allow is
    // not made: its barrier may still count the last one's bytes.  Rows of pages that are not there (no such row,
    // or a number outside the cache) are filled with zeros by the fetch.
    __device__ __forceinline__ void fetches(const Place& place, const CUtensorMap* km, const CUtensorMap* vm) const {
        const int lane = int(threadIdx.x) & 31;
        constexpr uint32_t SLOTS = C::SLOTS, RAWS = C::RAWS > 0 ? C::RAWS : 1;
        Walk walk = walk_from<C::ROWS, C::TN>(a, place);
        RunAt step;
        bool more = next_run<C::ROWS, C::TN>(a, walk, step);
        RunAt x = step;
        uint32_t runs = 0;
        publish(x, runs++, more, lane);
        if (lane == 0)
            a.meta[blockIdx.x] = more ? meta_of(place, x) : TreeMeta{0, place.chunk, 0, 0, 0, 0, place.lead};
        Look now{-1, 0};
        if (more) now = look(x, x.t0 * C::TN + lane * a.box);
        int it = 0;
        uint32_t n = 0, items = 0;  // tiles, and fetches of keys or values
        uint32_t fix_par = 0, fixed = 0;  // a bit for each slot: fix_full's parity, and whether it was used last
        for (bool on = true; more && on; ++n) {
            const uint32_t slot = n % SLOTS;
            const int tile = x.t0 + it, h = x.h;
            const bool part = (tile + 1) * C::TN > x.rq.len - x.rq.n;  // more than context rows
            // the next tile's pages: looked up before this one's fetch, but for a
            // run's first, as the fetch is not to wait for the walk
            const bool last = it + 1 == x.count;
            Look next{-1, 0};
            if (!last) next = look(x, (tile + 1) * C::TN + lane * a.box);
#pragma unroll 1
            for (int values = 0; values < 2; ++values, ++items) {
                const uint32_t r = items % RAWS;
                unsigned long long* bar = &sync->raw_full[r];
                uint32_t to = smem_addr(smem + C::RAW_AT) + r * C::RAW;
                if constexpr (C::kWide) {
                    if (n >= SLOTS)
                        bar_wait(values ? &sync->v_empty[slot] : &sync->k_empty[slot], (n / SLOTS - 1) & 1, sync);
                } else {
                    if (items >= RAWS) bar_wait(&sync->raw_empty[r], (items / RAWS - 1) & 1, sync);
                }
                // once a wait has given up, the place may be in use, or its last fetch under way
                on = !given_up();
                if (!on) break;
                if constexpr (C::kWide) {
                    to = smem_addr(smem) + (values ? C::V_AT + slot * C::V_SLOT : C::K_AT + slot * C::K_SLOT);
                    bar = values ? &sync->v_full[slot] : &sync->k_full[slot];
                    if (values) {
                        fixed = (fixed & ~(1u << slot)) | uint32_t(part) << slot;
                        fix_par ^= uint32_t(part) << slot;
                        if (part) bar = &sync->fix_full[slot];
                    }
                }
                fetch(values ? vm : km, values ? C::DV : C::DK, now, h, to, lane, bar);
            }
            if (C::kWide && lane == 0) sync->beat = n;
            ++it;
            if (last && on) {
                more = next_run<C::ROWS, C::TN>(a, walk, step);
                x = step;
                publish(x, runs++, more, lane);
                it = 0;
                if (more) next = look(x, x.t0 * C::TN + lane * a.box);
            }
            now = next;
        }
        // the block may not end before its fetches have, whether or not anyone still waits for them
        for (uint32_t k = items > 2 * SLOTS ? items - 2 * SLOTS : 0; C::kWide && k < items; ++k) {
            const uint32_t slot = k / 2 % SLOTS, par = (k / 2 / SLOTS) & 1;
            if (k % 2 == 0) landed(&sync->k_full[slot], par);
            else if (fixed >> slot & 1) landed(&sync->fix_full[slot], ~(fix_par >> slot) & 1);
            else landed(&sync->v_full[slot], par);
        }
        for (uint32_t k = items > RAWS ? items - RAWS : 0; !C::kWide && k < items; ++k)
            landed(&sync->raw_full[k % RAWS], (k / RAWS) & 1);
    }

    // For a whole warp, whose lanes may find `dead` at different times.
    __device__ __forceinline__ bool given_up() const { return __any_sync(0xffffffffu, sync->dead); }

    static __device__ __forceinline__ void landed(unsigned long long* b, uint32_t parity) {
        for (uint32_t i = 0; i < kSpins && !bar_test(b, parity); ++i) {
        }
    }

    // Where 16 bytes (8 lanes from 8 ch) of row `row` lie in a 16-bit tile.
    static __device__ __forceinline__ uint32_t line_at(int row, int ch) {
        return uint32_t(ch >> 3) * (C::TN * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
    }

    // Codes to fp16, in a tile's layout; rows from `valid` on become zeros.
    // Eight threads take 16 codes each of two successive rows: 64 of either row,
    // in an order that meets all banks both reading rows of codes and writing
    // lines (128 lanes: the second row's other half).  A team's step from one
    // such unit to the next is 4 or 8 rows modulo 8, so a thread's addresses
    // differ by constants from two places, and a unit costs a load, twelve
    // conversion instructions and two stores.  Two units a turn of a short loop:
    // unrolled (11 units) the helpers' code pushed the other roles' out of the
    // instruction cache, and 48 requests of 12000 fp8 rows took 354 us, not 273.
    template <int D>
    static __device__ __forceinline__ void widen(uint32_t raw, uint32_t to, int id, int valid) {
        constexpr int G = D / 64, UNITS = C::TN / 2 * G, STEP = kTeam / 8;
        constexpr int ROWS = STEP / G * 2;  // from a unit to the thread's next
        static_assert(STEP % G == 0 && ROWS % 4 == 0, "one of two places in the swizzle");
        const int u = id >> 3, odd = (id >> 2) & 1;
        const int row = u / G * 2 + odd, ch = ((G == 2 && odd ? u % G ^ 1 : u % G) << 2) + (id & 3);
        raw += row * D + ch * 16;
        // four rows on, chunk c of a line lies where c ^ 4 would
        constexpr int TURN = ROWS % 8 ? 4 : 0;
        uint32_t lo = to + line_at(row, 2 * ch), hi = to + line_at(row, 2 * ch + 1);
        uint32_t lo1 = to + line_at(row, (2 * ch) ^ TURN) + ROWS * 128;
        uint32_t hi1 = to + line_at(row, (2 * ch + 1) ^ TURN) + ROWS * 128;
        int left = UNITS - u;
        valid -= row;
#pragma unroll 1
        for (; left > 0; left -= 2 * STEP) {
            uint32_t w[2][4], h[8];
            lds128(w[0], raw);
            if (left > STEP) lds128(w[1], raw + ROWS * D);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i == 1 && left <= STEP) break;
                if (i * ROWS >= valid) w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0u;  // codes of 0
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[2 * j] = codes_to_half2<C::STORE, false>(w[i][j]);
                    h[2 * j + 1] = codes_to_half2<C::STORE, true>(w[i][j]);
                }
                sts128(i ? lo1 : lo, h[0], h[1], h[2], h[3]);
                sts128(i ? hi1 : hi, h[4], h[5], h[6], h[7]);
            }
            raw += 2 * ROWS * D;
            lo += 2 * ROWS * 128;
            hi += 2 * ROWS * 128;
            lo1 += 2 * ROWS * 128;
            hi1 += 2 * ROWS * 128;
            valid -= 2 * ROWS;
        }
    }

    // The values' team of e4m3: puts 0 in the place of codes of NaN in a tile's rows
    // [from, valid) (see add_not_finite).  A pass of its own, over the one or two
    // tiles of a request that have drafted rows: as a part of widen() it took 206 us
    // for 32 requests of 8000 rows and 64 query rows, and 190 so.
    __device__ __noinline__ void mend_codes(uint32_t raw, int id, int from, int valid, uint32_t run) const {
        bool found = false;
        for (int i = from * (C::DV / 16) + id; i < min(valid, C::TN) * (C::DV / 16); i += kTeam) {
            uint32_t w[4];
            lds128(w, raw + i * 16);
            if (take_out_nan4(w)) {
                found = true;
                sts128(raw + i * 16, w[0], w[1], w[2], w[3]);
            }
        }
        if (found) sync->patch[run & 7] = 1;
        __syncwarp();
        asm volatile("bar.sync 3, 96;" ::: "memory");
    }

    // 8-bit: the helpers turn codes into fp16 tiles and bring the scales, one
    // team keys (VALUES false), one values.
    template <bool VALUES>
    __device__ __forceinline__ void widen_tiles(int id) const {
        constexpr uint32_t SLOTS = C::SLOTS, RAWS = C::RAWS > 0 ? C::RAWS : 1;
        const float* scales = VALUES ? a.vs : a.ks;
        const int64_t* st = VALUES ? a.vs_st : a.ks_st;
        unsigned long long* full = VALUES ? sync->v_full : sync->k_full;
        unsigned long long* empty = VALUES ? sync->v_empty : sync->k_empty;
        constexpr int MORE = C::TN > kTeam ? 2 : 1;  // rows of a thread: id, and id + 96 for some
        const bool second = MORE == 2 && id < C::TN - kTeam;
        RunAt x;
        uint32_t n = 0, run = 0;
        constexpr bool MEND = VALUES && C::STORE == ROPE_CACHE_FP8;
        // (a team with a barrier of its own leaves together, see take_all)
        while (take_all<MEND ? 3 : 0, MEND ? kTeam : 32>(run, x)) {
            const int first = x.t0 * C::TN, prefix = x.rq.len - x.rq.n;
            Look now[MORE];
            now[0] = look(x, id < C::TN ? first + id : x.rq.len);
            if (MORE == 2) now[MORE - 1] = look(x, second ? first + kTeam + id : x.rq.len);
#pragma unroll 1
            for (int it = 0; it < x.count; ++it, ++n) {
                const uint32_t slot = n % SLOTS, item = 2 * n + (VALUES ? 1 : 0), r = item % RAWS;
                const int j0 = first + it * C::TN;
                float* sc = reinterpret_cast<float*>(smem + C::SC_AT + n % C::SCS * C::SC) + (VALUES ? C::TN : 0);
                float scale[MORE];
#pragma unroll
                for (int k = 0; k < MORE; ++k) {
                    scale[k] = 0.0f;
                    if (now[k].page >= 0 && now[k].page < a.pages)
                        scale[k] = __ldg(scales + now[k].page * st[0] + int64_t(now[k].off) * st[1] + int64_t(x.h) * st[2]);
                    const int j = j0 + C::TN + id + kTeam * k;
                    now[k] = look(x, (k ? second : id < C::TN) && it + 1 < x.count ? j : x.rq.len);
                }
                // In a ring of an odd number of places the team before in this
                // place was the other one: until it has emptied the place, the
                // parity of raw_full may still be that of the item before that.
                if (RAWS % 2 && item >= RAWS) bar_wait(&sync->raw_empty[r], (item / RAWS - 1) & 1, sync);
                bar_wait(&sync->raw_full[r], (item / RAWS) & 1, sync);
                if (n >= SLOTS) bar_wait(&empty[slot], (n / SLOTS - 1) & 1, sync);
                const uint32_t raw = smem_addr(smem + C::RAW_AT) + r * C::RAW;
                const uint32_t to = smem_addr(smem) + (VALUES ? C::V_AT + slot * C::V_SLOT : C::K_AT + slot * C::K_SLOT);
                if (MEND && j0 + C::TN > prefix) mend_codes(raw, id, max(prefix - j0, 0), x.rq.len - j0, run);
                widen<VALUES ? C::DV : C::DK>(raw, to, id, x.rq.len - j0);
                float most = 0.0f;
#pragma unroll
                for (int k = 0; k < MORE; ++k) {
                    float v = scale[k];
                    if (VALUES) {
                        // a drafted row's scale that is not finite is taken out (see add_not_finite)
                        if (j0 + id + kTeam * k >= prefix && !(fabsf(v) <= 3.4028234663852886e38f)) {
                            v = 0.0f;
                            sync->patch[run & 7] = 1;
                        }
                        most = fmaxf(most, v);
                    }
                    if (k ? second : id < C::TN) sc[id + kTeam * k] = v;
                }
                if (VALUES) {
                    // (scales are not negative: their bits order like them)
                    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
                    if ((id & 31) == 0) sc[C::TN + (id >> 5)] = __uint_as_float(bits);
                    if (id == 0) sc[C::TN + 3] = 0.0f;
                }
                to_async_proxy();
                bar_arrive(&sync->raw_empty[r]);
                bar_arrive(&full[slot]);
            }
            ++run;
        }
    }

    // 16-bit: in tiles with more than context rows, rows past the request's
    // become zeros (what the page holds there may be anything), and so do
    // drafted rows' values that are not finite (see add_not_finite).
    __device__ __forceinline__ void mend_tiles(int id) const {
        constexpr uint32_t SLOTS = C::SLOTS;
        RunAt x;
        uint32_t n = 0, run = 0, par = 0;  // a parity bit for each slot
        while (take_all<2, kHelpers, true>(run, x)) {
            const int prefix = x.rq.len - x.rq.n;
            for (int it = 0; it < x.count; ++it, ++n) {
                const int j0 = (x.t0 + it) * C::TN;
                if (j0 + C::TN <= prefix) continue;
                const uint32_t slot = n % SLOTS;
                bar_wait_run(&sync->fix_full[slot], (par >> slot) & 1, sync);
                par ^= 1u << slot;
                const uint32_t to = smem_addr(smem + C::V_AT) + slot * C::V_SLOT;
                const int from = max(prefix - j0, 0), valid = x.rq.len - j0;
                constexpr int CH = C::DV / 8;
                for (int i = from * CH + id; i < C::TN * CH; i += kHelpers) {
                    const int row = i / CH;
                    const uint32_t at = to + line_at(row, i % CH);
                    if (row >= valid) {
                        sts128(at, 0u, 0u, 0u, 0u);
                        continue;
                    }
                    uint32_t w[4];
                    lds128(w, at);
                    bool found = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool lo = not_finite<C::STORE>(w[j] & 0xffffu), hi = not_finite<C::STORE>(w[j] >> 16);
                        found = found || lo || hi;
                        w[j] = (lo ? 0u : w[j] & 0xffffu) | (hi ? 0u : w[j] & 0xffff0000u);
                    }
                    if (found) {
                        sts128(at, w[0], w[1], w[2], w[3]);
                        sync->patch[run & 7] = 1;
                    }
                }
                to_async_proxy();
                helpers_sync();
                if (id == 0) bar_arrive(&sync->v_full[slot]);
            }
            ++run;
        }
    }

    // ---------------------------------------------------------- products

    // The thread that issues the products.  A group's chain is s, (its
    // softmax), O; whichever group's next step is ready goes next.
    __device__ __forceinline__ void products() const {
        constexpr uint32_t QK = mma_shape<C::BF16, C::TN, false>();
        constexpr uint32_t PV = mma_shape<C::BF16, C::DV, true>();
        constexpr uint32_t SLOTS = C::SLOTS;
        const uint32_t q_at = smem_addr(smem), k_at = smem_addr(smem + C::K_AT), v_at = smem_addr(smem + C::V_AT);
        uint32_t before = 0, run = 0, q_par = 0, p_par = 0;  // p_par: a bit for each group
        RunAt x;
        while (take(run++, x)) {
            const int count = x.count;
            bar_wait(&sync->q_full, q_par, sync);
            q_par ^= 1;
            tmem_after();
            const int nv = C::PAIR ? 2 * count : count;  // steps; step v is group v & 1's
            // next steps of group w and of the other one
            int s_mine = 0, s_other = 1, p_mine = 0, p_other = 1, left = nv, w = 0;
            uint32_t spins = 0;
            // With an odd number of slots the tile before in a tile's slot is the
            // other group's: until that one's product is under way, the parity
            // of the slot's barrier may still be that of the tile before that.
            constexpr bool TURNS = !C::PAIR && SLOTS % 2;
            // (8-bit: rolled, for the instruction cache's sake, see widen; 16-bit pairs
            // took 118 us with this rolled and 105 without)
            constexpr int ISSUE = C::kWide ? 16 : 1;
            while (left > 0) {
                if (s_mine > p_mine && (!TURNS || p_other + 1 >= p_mine)) {
                    const int t = C::PAIR ? p_mine >> 1 : p_mine;
                    const uint32_t n = before + t, slot = n % SLOTS;
                    if (bar_poll(&sync->p_full[w], (p_par >> w) & 1) && bar_poll(&sync->v_full[slot], (n / SLOTS) & 1)) {
                        tmem_after();
                        const uint64_t vs = smem_matrix(v_at + slot * C::V_SLOT, C::TN * 128);
                        const uint32_t d = tmem + o_col(w), p = tmem + s_col(w);
                        const bool add = p_mine > 1;
#pragma unroll(ISSUE)
                        for (int k = 0; k < C::TN / 16; ++k) mma_ts(d, p + 8 * k, vs + k * (2048 >> 4), PV, add || k > 0);
                        p_par ^= 1u << w;
                        p_mine += 2;
                        // a pair's slot is free when both have been there
                        if (!C::PAIR || (p_other >> 1) > t) mma_commit(&sync->v_empty[slot]);
                        if (p_mine >= nv) mma_commit(&sync->o_full[w]);
                        --left;
                        spins = 0;
                    }
                }
                if (s_mine == p_mine && s_mine < nv && (!TURNS || s_other + 1 >= s_mine)) {
                    const int t = C::PAIR ? s_mine >> 1 : s_mine;
                    const uint32_t n = before + t, slot = n % SLOTS;
                    if (bar_poll(&sync->k_full[slot], (n / SLOTS) & 1)) {
                        tmem_after();
                        const uint64_t ks = smem_matrix(k_at + slot * C::K_SLOT, 16);
                        const uint64_t q = smem_matrix(q_at + (C::PAIR ? w * C::QTILE : 0), 16);
                        const uint32_t d = tmem + s_col(w);
#pragma unroll(ISSUE)
                        for (int k = 0; k < C::DK / 16; ++k)
                            mma_ss(d, q + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                                   ks + (((k >> 2) * (C::TN * 128) + (k & 3) * 32) >> 4), QK, k > 0);
                        mma_commit(&sync->s_full[w]);
                        s_mine += 2;
                        if (!C::PAIR || (s_other >> 1) > t) mma_commit(&sync->k_empty[slot]);
                        spins = 0;
                    }
                }
                if (++spins > kPolls || sync->dead) {
                    sync->dead = 1;
                    break;
                }
                // the other group's turn
                w ^= 1;
                const int s_ = s_mine, p_ = p_mine;
                s_mine = s_other;
                p_mine = p_other;
                s_other = s_;
                p_other = p_;
            }
            before += count;
        }
        mma_commit(&sync->done);
        for (uint32_t i = 0; i < kSpins && !bar_test(&sync->done, 0); ++i) {
        }
    }

    // ---------------------------------------------------------- softmax

    // The row tile's queries: 16-bit as they are, or fp16 in [-2, 2) with what
    // the row's s is multiplied by in `factor` (by row).  Eight lanes a row; rows
    // of a tile of 64 are stored once for each copy.
    __device__ __forceinline__ void stage_queries(const RunAt& x, int tid, float* factor) const {
        constexpr int N = C::DK / 64, EACH = 32;  // chunks of a lane; rows of the 256 threads
        constexpr int TOGETHER = C::ROWS / EACH < 4 ? C::ROWS / EACH : 4;
        const int sub = tid & 7;
#pragma unroll 1
        for (int r0 = tid >> 3; r0 < C::ROWS; r0 += EACH * TOGETHER) {
            uint4 y[TOGETHER][N];  // in flight together
#pragma unroll
            for (int i = 0; i < TOGETHER; ++i) {
                const int at = x.m * C::ROWS + r0 + EACH * i;
                const bool there = at < x.rq.n * a.G;
                uint32_t tok = 0, g = 0;
                if (there) a.div_group.divmod(uint32_t(at), tok, g);
                const uint4* src = reinterpret_cast<const uint4*>(a.q + int64_t(x.rq.qs + int(tok)) * a.q_st[0] +
                                                                  int64_t(x.h * a.G + int(g)) * a.q_st[1]);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int ch = 8 * k + sub;
                    y[i][k] = there && ch * 8 < a.Dk ? __ldg(src + ch) : make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < TOGETHER; ++i) {
                const int row = r0 + EACH * i;
                float down = 1.0f;
                if constexpr (!C::kWide) {
                    // the largest |q| of bit patterns: bf16 and fp16 order alike
                    uint32_t most = 0;
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const uint4 z = y[i][k];
                        most = max(most, max(max(z.x & 0x7fff0000u, z.y & 0x7fff0000u),
                                             max(z.z & 0x7fff0000u, z.w & 0x7fff0000u)) >> 16);
                        most = max(most, max(max(z.x & 0x7fffu, z.y & 0x7fffu), max(z.z & 0x7fffu, z.w & 0x7fffu)));
                    }
#pragma unroll
                    for (int d = 4; d; d /= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
                    const float big = a.bf16 ? __uint_as_float(most << 16)
                                             : __half2float(__ushort_as_half(static_cast<unsigned short>(most)));
                    const float p = row_power(__float_as_uint(big));
                    down = one_over_power(p);
                    if (sub == 0) factor[row] = row_factor(p, a.scale_log2);
                }
                const uint32_t to = smem_addr(smem) + (C::PAIR ? row / 128 * C::QTILE : 0) + row % 128 * 128 +
                                    ((sub ^ (row & 7)) << 4);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    uint4 z = y[i][k];
                    if constexpr (!C::kWide) {
                        float f[8];
                        widen8(z, a.bf16, f);
                        z = half8(f, down);
                    }
#pragma unroll
                    for (int copy = 0; copy < C::SPLIT; ++copy)
                        sts128(to + k * 16384 + copy * (C::ROWS * 128), z.x, z.y, z.z, z.w);
                }
            }
        }
    }


    // 32 scores of a row times the keys' scales.
    static __device__ __forceinline__ void scale32(float* s, const float* scale) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const float4 y = *reinterpret_cast<const float4*>(scale + j);
            const float2 lo = mul2(make_float2(s[j], s[j + 1]), make_float2(y.x, y.y));
            const float2 hi = mul2(make_float2(s[j + 2], s[j + 3]), make_float2(y.z, y.w));
            s[j] = lo.x;
            s[j + 1] = lo.y;
            s[j + 2] = hi.x;
            s[j + 3] = hi.y;
        }
    }

    // 32 scores in tensor memory: scaled (8-bit), and -inf where the bit is not set.
    static __device__ __forceinline__ void mask32(uint32_t at, const float* scale, uint32_t bits) {
        float s[32];
        tmem_ld32(s, at);
        tmem_wait_ld();
        tmem_here32(s);
        if constexpr (!C::kWide) scale32(s, scale);
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (!(bits >> j & 1u)) s[j] = -INFINITY;
        tmem_st32(at, reinterpret_cast<const uint32_t*>(s));
    }

    // The largest of 32 scales whose bit is set, and of u.
    static __device__ __noinline__ float largest_seen(const float* scale, uint32_t bits, float u) {
#pragma unroll 1
        for (int j = 0; j < 32; j += 4, bits >>= 4) {
            const float4 y = *reinterpret_cast<const float4*>(scale + j);
            u = fmaxf(fmaxf(fmaxf(u, bits & 1u ? y.x : 0.0f), bits & 2u ? y.y : 0.0f),
                      fmaxf(bits & 4u ? y.z : 0.0f, bits & 8u ? y.w : 0.0f));
        }
        return u;
    }

    static __device__ __forceinline__ float max_of32(const float* s) {
        float m[4] = {s[0], s[1], s[2], s[3]};  // four chains
#pragma unroll
        for (int j = 4; j + 8 <= 32; j += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = max3(m[i], s[j + 2 * i], s[j + 2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = fmaxf(m[i], s[28 + i]);
        return fmaxf(max3(m[0], m[1], m[2]), m[3]);
    }

    // The weights of 32 scores: their sum, and the 16-bit pairs at `to`.
    static __device__ __forceinline__ void weights32(const float* s, const float* scale, float factor, float base,
                                                     float2* sum, uint32_t to) {
        const float2 fac = make_float2(factor, factor), off = make_float2(base, base);
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            float2 e[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                e[i] = fma2(make_float2(s[j + 2 * i], s[j + 2 * i + 1]), fac, off);
                e[i].x = pow2(e[i].x);
                e[i].y = pow2(e[i].y);
                sum[i] = add2(sum[i], e[i]);
            }
            if constexpr (!C::kWide) {
                const float4 u = *reinterpret_cast<const float4*>(scale + j);
                e[0] = mul2(e[0], make_float2(u.x, u.y));
                e[1] = mul2(e[1], make_float2(u.z, u.w));
            }
            p[j / 2] = pack2<C::BF16>(e[0].x, e[0].y);
            p[j / 2 + 1] = pack2<C::BF16>(e[1].x, e[1].y);
        }
        tmem_st16(to, p);
    }

    // O of the thread's row times f.  The group's product before is complete: s
    // of this tile came after it.
    static __device__ __forceinline__ void rescale(uint32_t at, float f) {
#pragma unroll 1
        for (int c = 0; c < C::DV; c += 32) {
            float o[32];
            tmem_ld32(o, at + c);
            tmem_wait_ld();
            tmem_here32(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= f;
            tmem_st32(at + c, reinterpret_cast<const uint32_t*>(o));
        }
    }

    static __device__ __forceinline__ float exponent(float power) {  // of a power of two
        return float(int(__float_as_uint(power) >> 23) - 127);
    }

    __device__ __forceinline__ void softmax(int w) const {
        const int tid = int(threadIdx.x), row = tid & 127;
        const uint32_t lanes = tmem + (uint32_t(row & 96) << 16);  // this warp's lanes
        float2* ml = reinterpret_cast<float2*>(smem + C::ML_AT);
        RunAt x;
        uint32_t before = 0, run = 0, s_par = 0, o_par = 0;
        while (take_all<1, 256>(run, x)) {
            float* factors = reinterpret_cast<float*>(smem + C::FACTOR_AT);
            stage_queries(x, tid, factors);
            to_async_proxy();
            bar_arrive(&sync->q_full);

            const int rows = x.rq.n * a.G;
            // the thread's query row, and the columns of s that it sees to (of
            // 64 query rows each pair of warps has a copy, and its own columns)
            const int mine = C::PAIR ? row : row % C::ROWS, lo = row / (C::PAIR ? 128 : C::ROWS) * C::COLS;
            const int at = x.m * C::ROWS + (C::PAIR ? 128 * w : 0) + mine;
            const bool active = at - (row & 31) < rows;  // the warp has a row
            const int tok = min(int(a.div_group.div(uint32_t(at))), x.rq.n - 1);
            const int prefix = x.rq.len - x.rq.n, nv = C::PAIR ? 2 * x.count : x.count;
            float factor = a.scale_log2;
            if constexpr (!C::kWide) {
                groups_sync();
                factor = factors[(C::PAIR ? 128 * w : 0) + mine];
            }
            float m = -INFINITY, l = 0.0f, vref = 8.2718061255302767e-25f;  // 2^-80

#pragma unroll 1
            for (int v = w; v < nv; v += 2) {
                const int t = C::PAIR ? v >> 1 : v, j0 = (x.t0 + t) * C::TN;
                const uint32_t n = before + t;
                const float* sc = reinterpret_cast<const float*>(smem + C::SC_AT + n % C::SCS * C::SC);
                bar_wait(&sync->s_full[w], s_par, sync);
                __syncwarp();
                s_par ^= 1;
                tmem_after();
                if (active) {
                    const bool part = j0 + C::TN > prefix;  // more than context rows
                    float shrink = 1.0f;  // what l and O are multiplied by
                    float u = 0.0f;       // 8-bit: the largest scale of the values that the row sees
                    if constexpr (!C::kWide) {
                        // the scales came with the keys and the values
                        bar_wait(&sync->v_full[n % C::SLOTS], (n / C::SLOTS) & 1, sync);
                        __syncwarp();
                        if (!part) {
                            const float4 y = *reinterpret_cast<const float4*>(sc + 2 * C::TN);
                            u = fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w));
                        }
                    }
                    if (part) {
#pragma unroll 1
                        for (int c = lo; c < lo + C::COLS; c += 32) {
                            const uint32_t bits = sees32(a, x.rq.qs, tok, prefix, x.rq.len, j0 + c);
                            mask32(lanes + s_col(w) + c, sc + c, bits);
                            if constexpr (!C::kWide) u = largest_seen(sc + C::TN + c, bits, u);
                        }
                        tmem_wait_st();
                    }
                    if constexpr (!C::kWide) {
                        if (u > vref) {
                            const float p = power_above(u);
                            shrink = vref / p;
                            vref = p;
                        }
                    }
                    // s is held in registers by 16-bit rows, and by 8-bit pairs (whose rows
                    // have 64 lanes: 57 us against 62 when measured, for 2 requests of 131072 rows
                    // and 200 query rows).  Other 8-bit rows: it is read twice, 32 columns
                    // at a time, in loops small enough to stay in the instruction
                    // cache beside the helpers' (a batch of 48 requests of up to
                    // 12000 fp8 rows: 258 us, and 276 with s held).
                    constexpr int HELD = C::kWide || C::PAIR ? C::COLS : 32;
                    float s[HELD], top = -INFINITY;
                    const uint32_t from = lanes + s_col(w);
#pragma unroll 1
                    for (int c0 = lo; c0 < lo + C::COLS; c0 += HELD) {
#pragma unroll
                        for (int c = 0; c < HELD; c += 32) tmem_ld32(s + c, from + c0 + c);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < HELD; c += 32) {
                            tmem_here32(s + c);
                            if (!C::kWide && !part) scale32(s + c, sc + c0 + c);
                            top = fmaxf(top, max_of32(s + c));
                        }
                    }
                    top *= factor;
                    const bool up = top > m + C::kLag || (m == -INFINITY && top > m);
                    if (up) {
                        shrink *= pow2(m - top);
                        m = top;
                    }
                    // (both factors at once: a second rescale would read columns that the
                    // first one's stores, which are asynchronous, may not have reached)
                    if (__any_sync(0xffffffffu, shrink != 1.0f)) {
                        l *= shrink;
                        if (v > 1) rescale(lanes + o_col(w), shrink);
                    }
                    const float base = C::kBias - (m == -INFINITY ? 0.0f : m) - (C::kWide ? 0.0f : exponent(vref));
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll 1
                    for (int c0 = lo; c0 < lo + C::COLS; c0 += HELD) {
                        if constexpr (HELD < C::COLS) {
                            // (p of the columns before lies over s of columns before those)
                            tmem_ld32(s, from + c0);
                            tmem_wait_ld();
                            tmem_here32(s);
                            if (!part) scale32(s, sc + c0);
                        }
#pragma unroll
                        for (int c = 0; c < HELD; c += 32)
                            weights32(s + c, sc + C::TN + c0 + c, factor, base, sum, from + (c0 + c) / 2);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    if constexpr (C::SPLIT > 1) {
                        // weights of 0 in the columns of the other copies
                        const uint32_t none[16] = {};
#pragma unroll 1
                        for (int c = 0; c < C::TN; c += 32)
                            if (c < lo || c >= lo + C::COLS) tmem_st16(from + c / 2, none);
                    }
                    tmem_wait_st();
                }
                tmem_before();
                bar_arrive(&sync->p_full[w]);
            }
            if (w < nv) {
                bar_wait(&sync->o_full[w], o_par, sync);
                __syncwarp();
                o_par ^= 1;
                tmem_after();
            }
            if constexpr (!C::kWide) l *= vref;
            if constexpr (C::PAIR) finish(x, w, row, at, at < rows, active, m, l, vref, sync->patch[run & 7], lanes);
            else gather(x, w, row, active, nv, m, l, vref, &sync->patch[run & 7], ml, lanes);
            tmem_before();
            groups_sync();  // queries, O and ml are done with
            if (tid == 0) sync->patch[run & 7] = 0;
            before += x.count;
            ++run;
        }
    }

    // The results of a run of a pair.  A thread holds a row, which it would write
    // 16 bytes at a time, 32 rows an instruction; rows go through shared memory
    // (the queries' place; 32 words of 32 rows a warp, words swizzled by the
    // row), so that a warp writes 64 bytes of a row at once.  A part is written as
    // it is held, columns first.
    __device__ __forceinline__ void finish(const RunAt& x, int w, int row, int at, bool there, bool active, float m,
                                           float l, float vref, bool patch, uint32_t lanes) const {
        if (!active) return;
        const int lane = row & 31;
        const bool whole = x.slot < 0;
        OutAt to{nullptr, nullptr};
        float norm = C::kWide ? 1.0f : vref;
        if (there) {
            if (whole) {
                to = out_at(a, x.rq.qs, x.h, at);
                if (to.lse) *to.lse = lse_of(m, l, C::kBias);
                norm *= l == 0.0f ? 0.0f : 1.0f / l;  // a token that has seen no row gives zeros
            } else {
                a.part_ml[x.slot * C::ROWS + 128 * w + row] = make_float2(m, l);
            }
        }
        float* words = reinterpret_cast<float*>(smem + w * C::QTILE) + (row >> 5) * 1024;
#pragma unroll 1
        for (int c = 0; c < C::DV; c += 32) {
            float o[32];
            tmem_ld32(o, lanes + o_col(w) + c);
            tmem_wait_ld();
            tmem_here32(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= norm;
            if (patch && there) add_not_finite<C::STORE, C::TN, 32>(a, x, at, c, o);
            if (whole) {
                write32(words, o, to.out, c, lane);
            } else {
                // (rows that are not there have a place too)
                using P = PartAt<C::ROWS, C::DV>;
                float* part = a.part + P::block(x.slot, 4 * w + (row >> 5)) + c * 32 + lane;
#pragma unroll
                for (int j = 0; j < 32; ++j) part[j * 32] = o[j];
            }
        }
    }

    // The results of a run whose groups, and whose copies of the rows, each saw to
    // tiles and columns of their own: (m, l) and O of 2 SPLIT sources are joined
    // through shared memory (O in the queries' place, 16 columns at a time,
    // rows side by side).
    __device__ __forceinline__ void gather(const RunAt& x, int w, int row, bool active, int nv, float m, float l,
                                           float vref, const volatile uint32_t* patched, float2* ml,
                                           uint32_t lanes) const {
        constexpr int R = C::ROWS, SRC = 2 * C::SPLIT;
        const int tid = w * 128 + row, mine = row % R, src = w * C::SPLIT + row / R;
        const bool none = w >= nv;  // a group without a tile
        ml[src * R + mine] = none ? make_float2(-INFINITY, 0.0f) : make_float2(m, l);
        groups_sync();
        const bool patch = *patched != 0;  // (after both groups have waited for their products)
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < SRC; ++k) top = fmaxf(top, ml[k * R + mine].x);
        const float base = top == -INFINITY ? 0.0f : top;
        const float f = none ? 0.0f : pow2(m - base) * (C::kWide ? 1.0f : vref);
        const uint32_t words = smem_addr(smem), own = words + (src * 16 * R + mine) * 4;
        // the thread also writes four columns of the 16 of row tid % R (of R = 128,
        // eight), whose sums are the same all along
        const bool whole = x.slot < 0;
        const int r = tid % R, at = x.m * R + r, q0 = tid / R * 4;
        const bool writes = q0 < 16 && at < x.rq.n * a.G;
        float t = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < SRC; ++k) t = fmaxf(t, ml[k * R + r].x);
#pragma unroll
        for (int k = 0; k < SRC; ++k) {
            const float2 z = ml[k * R + r];
            sum += z.y * pow2(z.x - (t == -INFINITY ? 0.0f : t));
        }
        const float norm = sum == 0.0f ? 0.0f : 1.0f / sum;  // a token that has seen no row gives zeros
        char* out = nullptr;
        float* part = nullptr;
        if (writes) {
            if (whole) {
                const OutAt to = out_at(a, x.rq.qs, x.h, at);
                if (q0 == 0 && to.lse) *to.lse = lse_of(t, sum, C::kBias);
                out = to.out;
            } else {
                part = a.part + PartAt<R, C::DV>::block(x.slot, r / 32) + r % 32;
                if (q0 == 0) a.part_ml[x.slot * R + r] = make_float2(t, sum);
            }
        }
#pragma unroll 1
        for (int c = 0; c < C::DV; c += 16) {
            float o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = 0.0f;
            if (active && !none) {
                tmem_ld16(o, lanes + o_col(w) + c);
                tmem_wait_ld();
                tmem_here16(o);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(own + j * R * 4), "f"(o[j] * f) : "memory");
            groups_sync();
            if (writes) {
#pragma unroll
                for (int q = q0; q < 16; q += (R == 128 ? 8 : 16)) {
                    float z[SRC][4], y[4];
#pragma unroll
                    for (int k = 0; k < SRC; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            asm volatile("ld.shared.f32 %0, [%1];"
                                         : "=f"(z[k][j])
                                         : "r"(words + ((k * 16 + q + j) * R + r) * 4));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[j] = z[0][j];
#pragma unroll
                        for (int k = 1; k < SRC; ++k) y[j] += z[k][j];
                    }
                    if (patch) add_not_finite<C::STORE, C::TN, 4>(a, x, at, c + q, y);
                    if (out) {
                        if (c + q < a.Dv)
                            *reinterpret_cast<uint2*>(out + (c + q) * 2) =
                                a.bf16 ? make_uint2(pack2<true>(y[0] * norm, y[1] * norm), pack2<true>(y[2] * norm, y[3] * norm))
                                       : make_uint2(pack2<false>(y[0] * norm, y[1] * norm), pack2<false>(y[2] * norm, y[3] * norm));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[(c + q + j) * 32] = y[j];
                    }
                }
            }
            groups_sync();
        }
    }

    // The block's results, when one of its waits has given up: NaN in all of them,
    // those of the block's other runs too, and in its parts, whose joined results
    // then are NaN.  By the 256 threads of the softmax groups, after all roles.
    __device__ __noinline__ void give_up(const Place& place) const {
        const int tid = int(threadIdx.x);
        Walk walk = walk_from<C::ROWS, C::TN>(a, place);
        RunAt x;
        while (next_run<C::ROWS, C::TN>(a, walk, x)) {
            const int first = x.m * C::ROWS, left = min(C::ROWS, x.rq.n * a.G - first);
            if (x.slot >= 0) {
                for (int r = tid; r < C::ROWS; r += 256) a.part_ml[x.slot * C::ROWS + r] = make_float2(-INFINITY, NAN);
                continue;
            }
            for (int i = tid; i < left * (C::DV / 2); i += 256) {
                const int c = i % (C::DV / 2) * 2;
                const OutAt to = out_at(a, x.rq.qs, x.h, first + i / (C::DV / 2));
                if (c < a.Dv) *reinterpret_cast<uint32_t*>(to.out + c * 2) = 0x7fff7fffu;  // NaN of either type
                if (c == 0 && to.lse) *to.lse = NAN;
            }
        }
    }

    // 32 columns from c of the warp's rows; `mine` is the thread's own row's
    // place (null: none).
    __device__ __forceinline__ void write32(float* words, const float* o, char* mine, int c, int lane) const {
        const uint32_t at = smem_addr(words);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j) words[lane * 32 + (j ^ lane)] = o[j];
        __syncwarp();
        // two columns a lane, two rows an instruction, four of them at a time
        const int k = (lane & 15) * 2;
#pragma unroll 1
        for (int r0 = lane >> 4; r0 < 32; r0 += 8) {
            unsigned long long to[4];
            float y[4], z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + 2 * i;
                to[i] = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), r);
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(y[i]) : "r"(at + (r * 32 + (k ^ r)) * 4));
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(z[i]) : "r"(at + (r * 32 + ((k + 1) ^ r)) * 4));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (to[i] && c + k < a.Dv)
                    *reinterpret_cast<uint32_t*>(to[i] + (c + k) * 2) =
                        a.bf16 ? pack2<true>(y[i], z[i]) : pack2<false>(y[i], z[i]);
        }
        __syncwarp();
    }
};

// T: Tile<C>, or roles derived from it.
template <class T>
__global__ void __launch_bounds__(kTileThreads, 1)
rope_tree_tile_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap km,
                      const __grid_constant__ CUtensorMap vm) {
    using C = typename T::Cfg;
    extern __shared__ __align__(1024) char smem[];
    TileSync* sync = reinterpret_cast<TileSync*>(smem + C::SYNC_AT);
    const int warp = int(threadIdx.x) >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            // 16-bit: the fetch itself, or one helper for all; 8-bit: a team of helpers
            bar_init(&sync->k_full[i], C::kWide ? 1 : kTeam);
            bar_init(&sync->k_empty[i], 1);
            bar_init(&sync->v_full[i], C::kWide ? 1 : kTeam);
            bar_init(&sync->v_empty[i], 1);
            bar_init(&sync->fix_full[i], 1);
            bar_init(&sync->raw_full[i], 1);
            bar_init(&sync->raw_empty[i], kTeam);
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
        sync->runs = 0;
        sync->last = ~0u;
        sync->beat = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sync->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    after_predecessor();
    const Place place = find_place<C::ROWS, C::TN, kTileThreads>(a, reinterpret_cast<int64_t*>(smem));
    tmem_before();
    __syncthreads();
    tmem_after();
    const T tile{a, smem, sync, sync->tmem};

    // registers: 128 a thread at launch; 256 x 192 + 256 x 64 of the same 65536
    // (the host sees to it that the launch has them)
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        tile.softmax(warp >> 2);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 12) {
            if (threadIdx.x == 12 * 32) tile.products();
            __syncwarp();
        } else if (warp == 13) {
            tile.fetches(place, &km, &vm);
        } else {
            const int id = int(threadIdx.x) - (warp < 12 ? 256 : 320);
            if constexpr (C::kWide) tile.mend_tiles(id);
            else if (id < kTeam) tile.template widen_tiles<false>(id);
            else tile.template widen_tiles<true>(id - kTeam);
        }
    }
    tmem_before();
    __syncthreads();
    if (warp < 8 && sync->dead) tile.give_up(place);
    if (warp == 12) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sync->tmem));
    }
}

template <int STORE, int DK, int DV, int ROWS>
TreeKernel tile_kernel() {
    using C = TileCfg<STORE, DK, DV, ROWS>;
    return TreeKernel{reinterpret_cast<const void*>(&rope_tree_tile_kernel<Tile<C>>),
                      reinterpret_cast<const void*>(&rope_tree_join_kernel<C::ROWS, DV>), C::SMEM, kTileThreads,
                      C::TN, C::kBias, 256 * 192 + 256 * 64};
}

template <int STORE, int DK, int DV>
TreeKernel pick_tile_rows(const TreePlan& p) {
    if (p.rows <= 64) return tile_kernel<STORE, DK, DV, 64>();
    if constexpr (TileCfg<STORE, DK, DV, 128>::kWide || DK == 64)
        if (p.rows == 256) return tile_kernel<STORE, DK, DV, 256>();
    return tile_kernel<STORE, DK, DV, 128>();
}

}  // namespace rope
