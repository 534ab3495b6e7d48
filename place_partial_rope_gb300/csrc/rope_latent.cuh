// rope_latent.cuh -- attention of many query heads over a paged cache of latent rows (one
// row a token for all heads, whose first lanes are the value too), on tcgen05.
//
// Mathematics, with Q the query rows (tokens x heads) of a request and C its cache rows:
//     S^T = C Q^T    P^T = 2^(S^T scale - m)    O^T = V^T P^T,  V = C's first lanes
// in that transposed form: cache rows (and value lanes) are the 128 or 64 lanes of tensor
// memory, query rows its columns.  A row's 512 sums of O in fp32 fill a quarter of a
// lane's 512 columns so for 64 query rows (the other way round, 64 rows would use half of
// the lanes and all columns), few query rows (16 or 32 heads) make narrow, cheap
// products, and the two products take the same tile of C from shared memory: the first
// with the sum along its lines, the second with it across them.
//   The maximum that weights refer to may lag: it moves (and O and l shrink) when a score
// has passed it by more than 2^8, so that a tile costs one vote instead of a maximum over
// lanes.  `ref` is that maximum less a bias (7 for fp16 weights, which then stay between
// 2^-24 and 2^15); everything is counted from it.  Not rounded to a whole number: so the largest
// weight of the tile that has set it is a power of two, which 16 bits hold, and a row that
// outweighs the others comes out as it is (errors of single tokens over 20 rows 1.2 times those of
// the result's own rounding, and 1.45 with a whole number).  8-bit rows: the score has the row's
// scale u, the weight is 2^(s - ref) u and refers to the largest s + log2 u that the query
// row sees (u counted as 2^-80 at least there), so weights keep that range; l is
// the sum of 2^(s - ref).
//
// How.  One block an SM, 15 warps with a role each:
//   0-3   softmax.  A thread has 2 of a tile's 64 rows and every fourth pair of columns;
//         sums l stay in its registers for the whole run.  P^T goes to shared memory by
//         transposing stores.  O is read and written out when a run ends.
//   4, 14 issue tcgen05.mma: the scores', the values'.
//   5     fetches tiles by tensor copies (16-bit rows, pages of a multiple of 8 rows), and
//         walks the division of the work for all.
//   6-13  helpers: bring the queries of a run, and other tiles: 16-bit rows by
//         asynchronous copies, 8-bit rows as codes that become fp16 on the way.
// Two tiles of 64 rows x 576 lanes beside 64 query rows fill shared memory.
//   What bounds it: shared memory, which both products read at its full rate (1150 cycles for
// the scores of 64 query rows and 770 for the values of a tile of 64 rows, 570 more to bring it),
// and the chain of fetch, scores, softmax and values over two tiles in flight: 64 requests
// of 128 heads over 90 to 12000 bf16 rows take 161 us (2.9 TB/s; 68 by the cache's bytes), 3
// chunks of 200 to 256 tokens of 64 heads over 1031 to 4099 fp16 rows 396 us (606 TFLOP/s).  8-bit
// rows: threads that turn codes into fp16, and instruction fetch: 32 requests of 1 to 7 tokens
// of 32 heads over 8000 fp8 rows 179 us (352 TFLOP/s), 2 of 131072 int8 rows and 16 heads 74 us
// (2.0 TB/s).  One token of 16 heads over 4097 rows: 16 to 17 us, a tile a block and the join.
//   Every wait is bounded; one that gives up sets `dead`, the threads of a role leave
// together, and every result that the block has a share in becomes NaN.
#pragma once
#include "rope_latent.h"
#include "rope_tc.cuh"

namespace rope {

template <int STORE_, int ROWS_, bool BOXES_>
struct LatentCfg {
    static constexpr int STORE = STORE_, ROWS = ROWS_, TN = kLatentKeys;
    static constexpr bool BOXES = BOXES_;
    static constexpr bool kWide = STORE == ROPE_CACHE_BF16 || STORE == ROPE_CACHE_FP16;
    static constexpr bool BF16 = STORE == ROPE_CACHE_BF16;
    static constexpr int CHUNK = TN * 128;  // 64 lanes of a tile, in bytes
    static constexpr int CHUNKS = kLatentLanes / 64;
    // A tile in shared memory.  With tensor copies: its groups of chunks, one behind the other; of
    // four chunks the rows by eight, and of those the matrices of 8 x 64 lanes side by side; the
    // last group chunk by chunk.  So a copy can bring any number of eights of its lanes.
    // Without: all rows by eight.
    static constexpr int MATRIX = 1024;
    static constexpr uint32_t EIGHT = (BOXES ? 4 : CHUNKS) * MATRIX, EIGHT_LAST = BOXES ? MATRIX : EIGHT;
    static constexpr int Q_CHUNK = ROWS * 128, Q_BYTES = CHUNKS * Q_CHUNK;
    static constexpr int STAGE = CHUNKS * CHUNK, STAGES = 2;
    static constexpr int K_AT = Q_BYTES, P_AT = K_AT + STAGES * STAGE, SYNC_AT = P_AT + (ROWS < 64 ? ROWS * 256 : ROWS * 128);  // (P, and results turned over)
    static constexpr int kSmemMax = 232448;
    // Softmax groups of four warps, which share out the columns (query rows).  64 rows: two, and
    // four warps of helpers (ragged batch of 16-bit rows 194 us, and 181 so; chunks of prompts,
    // rows copied by threads, 657 and 569); 8-bit rows need all eight (182 us, with four 236).
    static constexpr int SG = ROWS == 64 && kWide ? 2 : 1, SR = ROWS / SG;
    static constexpr int HELPERS = SG == 2 ? 128 : 256, TEAM = HELPERS / 2;
    static constexpr float kBias = BF16 ? 0.0f : 7.0f, kLag = 8.0f;
    static constexpr int MORE = kWide ? 0 : (3 * ROWS + 2 * TN) * 4;  // factors and scales
    // tiles from one that is brought to one that is asked into L2 (2 to 4 do equally well,
    // none: ragged batch 161 -> 170 us)
    static constexpr int kAhead = 2;
    // tensor memory: O^T in tiles of 128 value lanes, then two S^T
    static constexpr uint32_t S_COL = 4 * ROWS;
};

// A try of a wait sleeps up to 20 us: fourteen warps that looked again and again would keep
// the two that issue products from their slots.
constexpr uint32_t kNaps = 1u << 17;  // tries of one wait before it gives up: 2.6 s

__device__ __forceinline__ bool bar_nap(unsigned long long* b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(smem_addr(b)), "r"(parity), "r"(20000u)
                 : "memory");
    return ok != 0;
}

struct LatentSync {
    // a tile's groups of lanes: brought, and done with
    unsigned long long full[2][3], empty[2][2], s_full[2], s_free[2], p_full, q_full[3], q_empty, run_full[3], done;
    uint32_t tmem;
    volatile uint32_t dead;
    volatile uint32_t patch[3][4];  // of run r at r % 3, by 128 value lanes: r + 1 when infinities were taken out
    volatile uint32_t taken;     // runs that the softmax has begun
    volatile uint32_t beat;      // tiles done
    RunAt run[3];                // run r at r % 3, when its barrier says so; of no tiles: there is none
    float red[256], fac[64];     // of the softmax
};

template <int ROWS>
__device__ __forceinline__ void latent_ld(float* r, uint32_t at) {
    if constexpr (ROWS == 64)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
            "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
            : ROPE_R8(r, 0), ROPE_R8(r, 8), ROPE_R8(r, 16), ROPE_R8(r, 24)
            : "r"(at)
            : "memory");
    else if constexpr (ROWS == 32)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
            "%14, %15}, [%16];"
            : ROPE_R8(r, 0), ROPE_R8(r, 8)
            : "r"(at)
            : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : ROPE_R8(r, 0)
                     : "r"(at)
                     : "memory");
}

template <int N>
__device__ __forceinline__ void latent_here(float* r) {
#pragma unroll
    for (int i = 0; i < N; i += 8) asm volatile("" : ROPE_B8(r, i));
}

// M x N, fp32 sums; A_MN: the first factor's lines run along its rows (values).
template <bool BF16, int M, int N, bool A_MN>
__host__ __device__ constexpr uint32_t latent_shape() {
    return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((A_MN ? 1u : 0u) << 15) |
           (uint32_t(N / 8) << 17) | (uint32_t(M / 16) << 24);
}

// The logarithm of the sum l 2^ref: l's powers of two are added to ref apart from the
// logarithm of its other part, which is below 1.
__device__ __forceinline__ float latent_lse(float ref, float l) {
    if (l == 0.0f) return -INFINITY;
    if (!(l >= 1.17549435e-38f && l <= 3.40282347e+38f)) return (ref + log2f(l)) * 0.69314718055994531f;
    const uint32_t bits = __float_as_uint(l);
    const float whole = ref + static_cast<float>(int(bits >> 23) - 127);
    return (whole + log2f(__uint_as_float((bits & 0x007fffffu) | 0x3f800000u))) * 0.69314718055994531f;
}

__device__ __forceinline__ uint32_t elected() {
    uint32_t me;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(me));
    return me;
}

// A product, and a commit, by the lane of the warp that has `me`.  a and b: the low words of
// the descriptors (see smem_matrix); EIGHT: bytes between a's groups of eight rows (b's are
// 1024), in the high words, which are constants.
template <uint32_t EIGHT>
__device__ __forceinline__ void mma_one(uint32_t me, uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool add) {
    constexpr uint64_t KIND = (uint64_t(1) << 46) | (uint64_t(2) << 61), A = KIND | (uint64_t(EIGHT >> 4) << 32),
                       B = KIND | (uint64_t(1024 >> 4) << 32);
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %5, 0;\nsetp.ne.b32 q, %4, 0;\n"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(A | a), "l"(B | b), "r"(shape), "r"(me), "r"(uint32_t(add))
                 : "memory");
}

__device__ __forceinline__ void commit_one(uint32_t me, unsigned long long* b) {
    asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_addr(b)),
                 "r"(me)
                 : "memory");
}

// Whether any of the 128 threads of softmax group `bar` - 1 says so.
__device__ __forceinline__ bool softmax_any(int bar, bool mine) {
    uint32_t any;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred q, %2, 128, p;\n"
                 "selp.u32 %0, 1, 0, q;\n}"
                 : "=r"(any)
                 : "r"(uint32_t(mine)), "r"(bar)
                 : "memory");
    return any != 0;
}

__device__ __forceinline__ void softmax_sync(int bar) { asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory"); }

template <class C>
struct Latent {
    using Cfg = C;
    const TreeArgs& a;
    char* smem;
    LatentSync* sync;
    uint32_t tmem;

    __device__ __forceinline__ int chunks() const { return latent_chunks(a); }
    __device__ __forceinline__ int value_tiles() const { return latent_value_tiles(a); }
    __device__ __forceinline__ int value_groups() const { return latent_value_groups(a); }
    __device__ __forceinline__ int groups() const { return latent_groups(a); }
    __device__ __forceinline__ int group_end(int g) const {
        return g < value_groups() ? min(4 * g + 4, chunks()) : chunks();
    }
    // Bytes of a tile before the group that begins with chunk c0 (or a later chunk of the last).
    static __device__ __forceinline__ uint32_t group_at(int c0) {
        return uint32_t(c0) * (C::BOXES ? C::CHUNK : C::MATRIX);
    }
    __device__ __forceinline__ uint32_t stage(uint32_t n) const { return smem_addr(smem + C::K_AT) + (n & 1) * C::STAGE; }

    // ---------------------------------------------------------- waits

    // False: it gave up, or another has.
    __device__ __forceinline__ bool wait(unsigned long long* b, uint32_t parity) const {
        if (bar_nap(b, parity)) return true;
        return wait_on(b, parity);
    }

    __device__ __noinline__ bool wait_on(unsigned long long* b, uint32_t parity) const {
        for (uint32_t i = 0; i < kNaps; ++i) {
            if (bar_nap(b, parity)) return true;
            if (sync->dead) return false;
        }
        sync->dead = 1;
        return false;
    }

    // For those that may rightly wait for a whole run: gives up when no tile has been
    // done between two such stretches.
    __device__ __forceinline__ void wait_run(unsigned long long* b, uint32_t parity) const {
        if (!bar_nap(b, parity)) wait_run_on(b, parity);
    }

    __device__ __noinline__ void wait_run_on(unsigned long long* b, uint32_t parity) const {
        for (uint32_t seen = ~0u;;) {
            for (uint32_t i = 0; i < kNaps; ++i) {
                if (bar_nap(b, parity)) return;
                if (sync->dead) return;
            }
            const uint32_t now = sync->beat;
            if (now == seen) break;
            seen = now;
        }
        sync->dead = 1;
    }

    __device__ __forceinline__ bool given_up() const { return __any_sync(0xffffffffu, sync->dead); }

    // Run r, when the block has one.
    __device__ __forceinline__ bool take(uint32_t r, RunAt& x) const {
        wait_run(&sync->run_full[r % 3], (r / 3) & 1);
        if (sync->dead) return false;
        x = sync->run[r % 3];
        return x.count > 0;
    }

    // For group g's place of tile n: values are free when the product with them is done,
    // the other lanes when the scores are.
    __device__ __forceinline__ bool wait_free(uint32_t n, int g) const {
        return n < 2 || wait(g < value_groups() ? &sync->empty[n & 1][g] : &sync->s_full[n & 1], (n / 2 - 1) & 1);
    }

    // Until the last product of tile n is done.
    __device__ __forceinline__ void wait_product(uint32_t n) const {
        wait(&sync->empty[n & 1][value_groups() - 1], (n / 2) & 1);
    }

    // ---------------------------------------------------------- the walk, and tensor copies

    // The block's next run.  Of two blocks that walk a pair of row tiles (blockIdx.y) each has one.
    __device__ __forceinline__ bool run_after(LatentWalk& walk, RunAt& x) const {
        if (!next_run<C::ROWS, C::TN>(a, walk, x)) return false;
        x.m = x.m * int(gridDim.y) + int(blockIdx.y);
        if (x.slot >= 0) x.slot += int64_t(blockIdx.y) * 2 * gridDim.x;
        return true;
    }

    // Run r for the other roles, when all of them have taken run r - 3, whose place it gets.  With
    // tensor copies that is so: the copies before it were made when the products of the tile two
    // before them, and so of run r - 3, were done.  Else it is waited for: where one softmax group
    // has taken a run, every role has been through the run before that.
    __device__ __forceinline__ void publish(RunAt& x, uint32_t r, bool there, int lane) const {
        if (lane == 0) {
            if constexpr (!C::BOXES) {
                uint32_t seen = ~0u, i = 0;
                while (r >= sync->taken + 2 && !sync->dead) {
                    __nanosleep(200);
                    if (++i == kSpins) {
                        i = 0;
                        if (sync->beat == seen) sync->dead = 1;
                        seen = sync->beat;
                    }
                }
            }
            if (!there) x.count = 0;
            sync->run[r % 3] = x;
            bar_arrive(&sync->run_full[r % 3]);
        }
        __syncwarp();
    }

    // Where a.box rows of a tile lie, all in one page.
    struct Box {
        int page, off;  // page -1: no such rows
    };

    __device__ __forceinline__ Box box_of(const RunAt& x, int tile, int lane) const {
        Box r{-1, 0};
        const int j = tile * C::TN + lane * a.box;
        if (j < x.rq.len) {
            uint32_t p, off;
            a.div_page.divmod(uint32_t(j), p, off);
            r.off = int(off);
            r.page = __ldg(a.table + int64_t(x.r) * a.table_stride + p);
        }
        return r;
    }

    __device__ __forceinline__ void fetches(const Place& place, const LatentMaps& maps) const {
        const int lane = int(threadIdx.x) & 31, all = groups();
        LatentWalk walk = latent_walk_from<C::ROWS, C::TN>(a, place);
        RunAt x;
        uint32_t run = 0, n = 0, copies = 0;  // runs, tiles, groups of them asked for
        bool first = true;
        for (;; ++run) {
            const bool there = run_after(walk, x);
            if (first && lane == 0 && blockIdx.y == 0)
                a.meta[blockIdx.x] = there ? meta_of(place, walk, x) : TreeMeta{0, place.chunk, 0, 0, 0, 0, 0};
            first = false;
            publish(x, run, there, lane);
            if (!there || given_up()) break;
            if constexpr (C::BOXES) {
                // a lane a box, looked up a tile ahead; rows that are not there are filled with zeros
                const int boxes = C::TN / a.box;
                Box now{-1, 0};
                if (lane < boxes) now = box_of(x, x.t0, lane);
                bool on = true;
                for (int it = 0; on && it < x.count; ++it, ++n) {
                    Box next{-1, 0};
                    if (it + 1 < x.count && lane < boxes) next = box_of(x, x.t0 + it + 1, lane);
                    const uint32_t to = stage(n);
                    for (int g = 0, c = 0; g < all; ++g) {
                        // where a wait has given up, the place may be in use, or its last copy under way
                        on = __all_sync(0xffffffffu, wait_free(n, g));
                        if (!on) break;
                        const uint32_t bar = smem_addr(&sync->full[n & 1][g]);
                        const bool values = g < value_groups();
                        const int end = values ? c + 4 : chunks(), each = values ? 4 : 1;  // (chunks past a row: zeros)
                        if (lane == 0)
                            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                                         "r"((end - c) * C::CHUNK)
                                         : "memory");
                        __syncwarp();
                        ++copies;
                        if (lane < boxes)
                            for (int i = c; i < end; i += each)
                                asm volatile(
                                    "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                                    "[%0], [%1, {%2, %2, %3, %4, %5}], [%6];" ::"r"(
                                        to + i * C::CHUNK + lane * (a.box >> 3) * each * C::MATRIX),
                                    "l"(values ? &maps.four : &maps.one), "r"(0), "r"(i), "r"(now.off >> 3),
                                    "r"(now.page), "r"(bar)
                                    : "memory");
                        c = end;
                    }
                    // a later tile is on its way from memory to L2 meanwhile (in small boxes that costs
                    // more than it gives: ragged batch in boxes of 8 rows 187 us, and 251 so)
                    if (boxes == 1 && lane == 0 && it + C::kAhead < x.count) {
                        const Box far = box_of(x, x.t0 + it + C::kAhead, 0);
                        if (far.page >= 0 && far.page < a.pages)
                            for (int c = 0; c < chunks(); c += 4)
                                asm volatile("cp.async.bulk.prefetch.tensor.5d.L2.global.tile [%0, {%1, %1, %2, %3, %4}];" ::"l"(
                                                 &maps.four), "r"(0), "r"(c), "r"(far.off >> 3), "r"(far.page)
                                             : "memory");
                    }
                    now = next;
                }
            }
        }
        // the block may not end before its copies have, whether or not anyone still waits for them
        if constexpr (C::BOXES)
            for (uint32_t k = copies > 2u * all ? copies - 2 * all : 0; k < copies; ++k)
                for (uint32_t i = 0; i < kSpins && !bar_test(&sync->full[k / all & 1][k % all], (k / all / 2) & 1); ++i) {
                }
    }

    // ---------------------------------------------------------- helpers

    // Where 16 bytes (8 lanes from 8 piece) of query row `row` lie.
    static __device__ __forceinline__ uint32_t line_at(int row, int piece) {
        return uint32_t(piece >> 3) * C::Q_CHUNK + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
    }

    // The queries of a run: eight threads a row.
    __device__ __forceinline__ void queries(const RunAt& x, uint32_t run, int id) const {
        const int first = x.m * C::ROWS, left = min(C::ROWS, x.rq.n * a.G - first);
        const uint32_t to = smem_addr(smem);
        const int pieces = a.Dk / 8;
        if constexpr (C::kWide) {
            for (int row = id >> 3; row < C::ROWS; row += C::HELPERS / 8) {
                const char* src = nullptr;
                if (row < left) {
                    uint32_t tok, g;
                    a.div_group.divmod(uint32_t(first + row), tok, g);
                    src = a.q + int64_t(x.rq.qs + int(tok)) * a.q_st[0] + int64_t(g) * a.q_st[1];
                }
                for (int c = 0; c < chunks(); ++c) {
                    const int piece = c * 8 + (id & 7);
                    const bool ok = src && piece < pieces;
                    copy16(to + line_at(row, piece), ok ? src + piece * 16 : a.q, ok);
                }
            }
            copies_commit();
            copies_wait<0>();
        } else {
#pragma unroll 1
            for (int row = id >> 3; row < C::ROWS; row += C::HELPERS / 8) {
                const char* src = nullptr;
                if (row < left) {
                    uint32_t tok, g;
                    a.div_group.divmod(uint32_t(first + row), tok, g);
                    src = a.q + int64_t(x.rq.qs + int(tok)) * a.q_st[0] + int64_t(g) * a.q_st[1];
                }
                uint4 w[C::CHUNKS];
#pragma unroll
                for (int c = 0; c < C::CHUNKS; ++c) {
                    const int piece = c * 8 + (id & 7);
                    w[c] = src && piece < pieces ? __ldg(reinterpret_cast<const uint4*>(src) + piece)
                                                 : make_uint4(0, 0, 0, 0);
                }
                uint32_t most = 0;
                float f[8];
#pragma unroll
                for (int c = 0; c < C::CHUNKS; ++c) {
                    widen8(w[c], a.bf16, f);
                    most = max(most, most_of(f));
                }
#pragma unroll
                for (int d = 1; d < 8; d *= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
                const float p = row_power(most), by = one_over_power(p);
                if ((id & 7) == 0) factors(run)[row] = row_factor(p, a.scale_log2);
#pragma unroll
                for (int c = 0; c < C::CHUNKS; ++c) {
                    widen8(w[c], a.bf16, f);
                    w[c] = half8(f, by);
                }
#pragma unroll
                for (int c = 0; c < C::CHUNKS; ++c)
                    sts128(to + line_at(row, c * 8 + (id & 7)), w[c].x, w[c].y, w[c].z, w[c].w);
            }
        }
    }

    // 8-bit: the factors of a run's query rows, and the scales of a tile's rows.  Those of run r
    // are written when the scores of run r - 1 are done, which may be two tiles (and runs)
    // ahead of what the softmax has read: three places.
    __device__ __forceinline__ float* factors(uint32_t run) const {
        return reinterpret_cast<float*>(smem + C::SYNC_AT + sizeof(LatentSync)) + run % 3 * C::ROWS;
    }
    __device__ __forceinline__ float* scales(uint32_t n) const {
        return reinterpret_cast<float*>(smem + C::SYNC_AT + sizeof(LatentSync)) + 3 * C::ROWS + (n & 1) * C::TN;
    }

    // A cache row: its bytes, and its scale.
    struct Row {
        const char* p;  // null: there is none
        float scale;
    };

    __device__ __forceinline__ Row row_of(const RunAt& x, int j) const {
        Row r{nullptr, 0.0f};
        if (j < x.rq.len) {
            uint32_t p, off;
            a.div_page.divmod(uint32_t(j), p, off);
            const int page = __ldg(a.table + int64_t(x.r) * a.table_stride + p);
            if (page >= 0 && page < a.pages) {
                r.p = a.k + page * a.k_st[0] + int64_t(off) * a.k_st[1];
                if constexpr (!C::kWide) r.scale = __ldg(a.ks + page * a.ks_st[0] + int64_t(off) * a.ks_st[1]);
            }
        }
        return r;
    }

    // A tile without tensor copies, by the threads of a team: eight a row, four rows a thread
    // at a time.
    __device__ __forceinline__ bool load(const RunAt& x, int it, uint32_t n, int tid) const {
        constexpr int STEP = C::TEAM / 8, PASSES = C::TN / (4 * STEP);
        const int sub = tid & 7, pieces = a.Dk / 8, all = groups();
        const uint32_t to = stage(n);
#pragma unroll 1
        for (int pass = 0; pass < PASSES; ++pass) {
            const int row = pass * 4 * STEP + (tid >> 3);
            const uint32_t at = to + (row >> 3) * C::EIGHT + (row & 7) * 128 + ((sub ^ (row & 7)) << 4),
                           step = STEP / 8 * C::EIGHT;
            Row r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = row_of(x, (x.t0 + it) * C::TN + row + STEP * i);
#pragma unroll 1
            for (int g = 0, c = 0; g < all; ++g) {
                const int end = group_end(g);
                if constexpr (C::kWide) {
                    if (pass == 0 && !__all_sync(0xffffffffu, wait_free(n, g))) {
                        copies_wait<0>();
                        return false;
                    }
#pragma unroll 1
                    for (; c < end; ++c) {
                        const int piece = c * 8 + sub;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bool ok = r[i].p && piece < pieces;
                            copy16(at + c * C::MATRIX + i * step, ok ? r[i].p + piece * 16 : a.k, ok);
                        }
                    }
                    copies_commit();
                } else {
                    // codes are asked for before the place is free, and become fp16 on their way
                    bool waited = pass > 0;
#pragma unroll 1
                    for (; c < end; c = min(c + 4, end)) {
                        uint2 w[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int piece = (c + k) * 8 + sub;
                                w[i][k] = r[i].p && c + k < end && piece < pieces
                                              ? __ldg(reinterpret_cast<const uint2*>(r[i].p) + piece)
                                              : make_uint2(0, 0);
                            }
                        if (!waited && !__all_sync(0xffffffffu, wait_free(n, g))) return false;
                        waited = true;
                        // (the scales of tile n - 2 have been read when its first product is done)
                        if (c == 0 && sub == 0)
#pragma unroll
                            for (int i = 0; i < 4; ++i) scales(n)[row + STEP * i] = r[i].scale;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (c + k < end)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    sts128(at + (c + k) * C::MATRIX + i * step,
                                           codes_to_half2<C::STORE, false>(w[i][k].x),
                                           codes_to_half2<C::STORE, true>(w[i][k].x),
                                           codes_to_half2<C::STORE, false>(w[i][k].y),
                                           codes_to_half2<C::STORE, true>(w[i][k].y));
                    }
                    if (pass + 1 == PASSES) {
                        to_async_proxy();
                        bar_arrive(&sync->full[n & 1][g]);
                    }
                }
            }
        }
        if constexpr (C::kWide)  // groups as they come
            for (int g = 0; g < all; ++g) {
                if (all - g == 3) copies_wait<2>();
                else if (all - g == 2) copies_wait<1>();
                else copies_wait<0>();
                to_async_proxy();
                bar_arrive(&sync->full[n & 1][g]);
            }
        return true;
    }

    // Queries of all runs and, without tensor copies, their tiles: two teams, one for
    // either of the tiles' places, so that both are on their way at a time.  A team's first tile
    // of a run comes before the queries, which have to wait for the scores of the run before.
    __device__ __forceinline__ void help(int id) const {
        const uint32_t team = uint32_t(id) / C::TEAM;
        uint32_t n0 = 0;  // tiles of the runs before
        for (uint32_t run = 0;; ++run) {
            RunAt x;
            if (!__all_sync(0xffffffffu, take(run, x))) return;
            const int first = int((n0 ^ team) & 1);
            if constexpr (!C::BOXES)
                if (first < x.count && !load(x, first, n0 + first, id % C::TEAM)) return;
            if (run > 0) wait_run(&sync->q_empty, (run - 1) & 1);
            if (given_up()) return;
            queries(x, run, id);
            to_async_proxy();
            bar_arrive(&sync->q_full[run % 3]);
            if constexpr (!C::BOXES)
                for (int it = first + 2; it < x.count; it += 2)
                    if (!load(x, it, n0 + it, id % C::TEAM)) return;
            n0 += x.count;
        }
    }

    // ---------------------------------------------------------- products

    // Two warps issue products, one the scores', one the values': neither waits for what
    // the other needs.  A whole warp goes through the loops, so that descriptors stay in
    // uniform registers, and one lane issues: 30 to 38 cycles a product, where a lane alone
    // took 43 and more (67, forming each descriptor anew), and the tensor pipe takes 23 to 32
    // for the scores' and 39 to 48 for the values'.

    __device__ __forceinline__ void scores() const {
        constexpr uint32_t shape = latent_shape<C::BF16, C::TN, C::ROWS, false>();
        const uint32_t me = elected(), q = __shfl_sync(0xffffffffu, smem_addr(smem) >> 4, 0);
        const int all = chunks(), last = min(4 * value_groups(), all), groups_of_values = value_groups();
        uint32_t n = 0;
        for (uint32_t run = 0;; ++run) {
            RunAt x;
            if (!__all_sync(0xffffffffu, take(run, x))) break;
            const int count = __shfl_sync(0xffffffffu, x.count, 0);
            wait(&sync->q_full[run % 3], (run / 3) & 1);
            bool on = true;
            for (int it = 0; on && it < count; ++it, ++n) {
                // the softmax has read the scores before the last
                if (n >= 2) wait(&sync->s_free[n & 1], (n / 2 - 1) & 1);
                tmem_after();
                const uint32_t to = __shfl_sync(0xffffffffu, tmem + C::S_COL + (n & 1) * C::ROWS, 0);
                const uint32_t k = __shfl_sync(0xffffffffu, stage(n) >> 4, 0), par = (n / 2) & 1;
                unsigned long long* full = sync->full[n & 1];
                int c = 0;
#pragma unroll 1
                for (; c < last; ++c) {
                    if (c % 4 == 0) on = wait(full + c / 4, par);
                    const uint32_t x0 = k + (group_at(c & ~3) >> 4) + (c & 3) * (C::MATRIX >> 4),
                                   y0 = q + c * (C::Q_CHUNK >> 4);
                    mma_one<C::EIGHT>(me, to, x0, y0, shape, c > 0);
#pragma unroll
                    for (int i = 1; i < 4; ++i) mma_one<C::EIGHT>(me, to, x0 + i * 2, y0 + i * 2, shape, true);
                }
                if (c < all) on = wait(full + groups_of_values, par);
#pragma unroll 1
                for (; c < all; ++c) {
                    const uint32_t x0 = k + (group_at(c) >> 4), y0 = q + c * (C::Q_CHUNK >> 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_one<C::EIGHT_LAST>(me, to, x0 + i * 2, y0 + i * 2, shape, true);
                }
                on = __all_sync(0xffffffffu, on);  // (given up: the scores are whatever they are)
                commit_one(me, &sync->s_full[n & 1]);
                if (it + 1 == count) commit_one(me, &sync->q_empty);
            }
            if (given_up()) break;
        }
        commit_one(me, &sync->done);
    }

    __device__ __forceinline__ void products() const {
        constexpr uint32_t shape = latent_shape<C::BF16, 128, C::ROWS, true>();
        constexpr uint32_t lead = uint32_t(C::MATRIX >> 4) << 16;  // from 64 value lanes to the next
        const uint32_t me = elected(), p = __shfl_sync(0xffffffffu, smem_addr(smem + C::P_AT) >> 4, 0);
        const int tiles = value_tiles();
        uint32_t n = 0;
        for (uint32_t run = 0;; ++run) {
            RunAt x;
            if (!__all_sync(0xffffffffu, take(run, x))) break;
            const int count = __shfl_sync(0xffffffffu, x.count, 0);
            bool on = true;
            for (int it = 0; on && it < count; ++it, ++n) {
                on = __all_sync(0xffffffffu, wait(&sync->p_full, n & 1));
                tmem_after();
                const uint32_t v = __shfl_sync(0xffffffffu, (stage(n) >> 4) | lead, 0);
                const uint32_t to = __shfl_sync(0xffffffffu, tmem, 0);
#pragma unroll 1
                for (int t = 0; t < tiles; ++t) {
                    const uint32_t v0 = v + (group_at(t >> 1 << 2) >> 4) + (t & 1) * (C::MATRIX >> 3);
                    mma_one<C::EIGHT>(me, to + t * C::ROWS, v0, p, shape, it > 0);
#pragma unroll
                    for (int i = 1; i < 4; ++i)
                        mma_one<C::EIGHT>(me, to + t * C::ROWS, v0 + i * (C::EIGHT >> 3), p + i * 2, shape, true);
                    if (t % 2 == 1 || t + 1 == tiles) commit_one(me, &sync->empty[n & 1][t / 2]);
                }
                if (me) sync->beat = n + 1;
            }
            if (given_up()) break;
        }
        commit_one(me, &sync->done);
    }

    // Tensor memory may not go before the last product has.
    __device__ __forceinline__ void all_done() const {
        for (uint32_t i = 0; i < kSpins && !bar_test(&sync->done, 0); ++i) {
        }
        __syncwarp();
    }

    // ---------------------------------------------------------- softmax

    // The last tiles of a request: values of rows that are not there become zeros, and
    // those of drafted rows that are not finite are taken out: a weight of 0 times them
    // would reach the tokens that do not see the row.  Of those that do see it, a NaN (the row is
    // their key, too) has made the score and all results NaN, but infinities may have
    // made a score of -inf, and are put back (see finish).
    __device__ __noinline__ void mend(uint32_t n, int from, int valid, uint32_t run, int group) const {
        const int pieces = min(value_tiles() * 16, chunks() * 8), lane = int(threadIdx.x) & 31;
        uint32_t found = 0;  // infinities, by 128 lanes
        for (int row = from + (int(threadIdx.x) >> 5 & 3) * C::SG + group; row < C::TN; row += 4 * C::SG)
            for (int piece = lane; piece < pieces; piece += 32) {
                const int c0 = piece >> 5 << 2;  // its group's first chunk
                const uint32_t at = stage(n) + group_at(c0) + (row >> 3) * C::EIGHT + ((piece >> 3) - c0) * C::MATRIX +
                                    (row & 7) * 128 + (((piece & 7) ^ (row & 7)) << 4);
                if (row >= valid) {
                    sts128(at, 0, 0, 0, 0);
                    continue;
                }
                uint32_t w[4], bad = 0;
                lds128(w, at);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    constexpr int KIND = C::BF16 ? ROPE_CACHE_BF16 : ROPE_CACHE_FP16;
                    if (not_finite<KIND>(w[j])) w[j] &= 0xffff0000u, bad = 1;
                    if (not_finite<KIND>(w[j] >> 16)) w[j] &= 0xffffu, bad = 1;
                }
                if (bad) {
                    if constexpr (C::kWide) {
                        constexpr uint32_t INF = C::BF16 ? 0x7f80u : 0x7c00u;
                        uint32_t was[4];
                        lds128(was, at);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if ((was[j] & 0x7fffu) == INF || (was[j] >> 16 & 0x7fffu) == INF) found |= 1u << (piece >> 4);
                    }
                    sts128(at, w[0], w[1], w[2], w[3]);
                }
            }
        if (found)
            for (int t = 0; t < 4; ++t)
                if (found >> t & 1u) sync->patch[run % 3][t] = run + 1;
        __syncwarp();
    }

    // A group's columns of O times the factors of their rows.
    __device__ __forceinline__ void shrink(uint32_t lanes, int col0) const {
        const int tiles = value_tiles();
#pragma unroll 1
        for (int i = 0; i < tiles * C::SR; i += 16) {
            const int c = i / C::SR * C::ROWS + col0 + i % C::SR;
            float o[16];
            tmem_ld16(o, lanes + c);
            tmem_wait_ld();
            tmem_here16(o);
            const float* f = sync->fac + c % C::ROWS;
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * f[k]);
            tmem_st16(lanes + c, w);
        }
        tmem_wait_st();
    }

    // Two columns (i even) of s scale - ref (8-bit: s u times the row's factor, less ref).
    // 16-bit: what is not seen is -inf in s already; 8-bit: it becomes so here, as the scale
    // may have any sign.
    __device__ __forceinline__ float2 from_reference(const float* s, const float* ref, const float* qf, const float* u,
                                                     uint32_t seen, int i) const {
        const int c = (i >> 2) * 2, h = (i >> 1) & 1;
        const float2 r = make_float2(-ref[c], -ref[c + 1]);
        float2 y = make_float2(s[i], s[i + 1]);
        if constexpr (C::kWide) return fma2(y, make_float2(a.scale_log2, a.scale_log2), r);
        y = fma2(mul2(y, make_float2(u[h], u[h])), make_float2(qf[c], qf[c + 1]), r);
        if (!(seen >> i & 1u)) y.x = -INFINITY;
        if (!(seen >> i & 2u)) y.y = -INFINITY;
        return y;
    }

    __device__ __forceinline__ void softmax(int group) const {
        constexpr int NC = C::SR / 4, J = C::SR / 8;  // columns of a thread, blocks of eight
        const int tid = int(threadIdx.x) & 127, lane = tid & 31, warp = tid >> 5, k0 = warp * 16 + (lane >> 2),
                  col0 = group * C::SR, c0 = col0 + (lane & 3) * 2, bar = group + 1;
        float* red = sync->red + group * 4 * C::SR;  // the warps' maxima of the group's columns
        const uint32_t lanes = tmem + (uint32_t(warp * 32) << 16);
        // of the four 8 x 8 matrices of a transposing store, this thread names a line
        const int mat = lane >> 3, qrow = col0 + (mat >> 1) * 8 + (lane & 7), chunk = warp * 2 + (mat & 1);
        const uint32_t p_at = smem_addr(smem + C::P_AT) + qrow * 128 + ((chunk ^ (qrow & 7)) << 4);
        RunAt x;
        uint32_t n = 0;
        for (uint32_t run = 0;; ++run) {
            if (softmax_any(bar, !take(run, x))) return;
            if (threadIdx.x == 0) sync->taken = run + 1;
            const int prefix = x.rq.len - x.rq.n, first = x.m * C::ROWS;
            float ref[NC], l[NC], qf[C::kWide ? 1 : NC];
#pragma unroll
            for (int i = 0; i < NC; ++i) ref[i] = -3.40282347e+38f, l[i] = 0.0f;
            for (int it = 0; it < x.count; ++it, ++n) {
                const int tile = x.t0 + it;
                const bool part = (tile + 1) * C::TN > prefix;  // more than context rows
                float s[C::SR / 2], u[2] = {1.0f, 1.0f}, lu[2] = {0.0f, 0.0f};
                wait(&sync->s_full[n & 1], (n / 2) & 1);
                if (part || !C::kWide)  // what copies or helpers wrote is seen
                    for (int g = 0; g < value_groups(); ++g) wait(&sync->full[n & 1][g], (n / 2) & 1);
                __syncwarp();
                tmem_after();
                latent_ld<C::SR>(s, lanes + C::S_COL + (n & 1) * C::ROWS + col0);
                if constexpr (!C::kWide) {
                    if (it == 0) wait(&sync->q_full[run % 3], (run / 3) & 1);  // the helpers' factors are seen
                    if (it == 0)
#pragma unroll
                        for (int i = 0; i < NC; ++i) qf[i] = factors(run)[(i >> 1) * 8 + c0 + (i & 1)];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        u[i] = scales(n)[k0 + 8 * i];
                        lu[i] = log2f(fmaxf(fabsf(u[i]), 8.2718061255302767e-25f));  // 2^-80
                    }
                }
                tmem_wait_ld();
                latent_here<C::SR / 2>(s);
                tmem_before();
                bar_arrive(&sync->s_free[n & 1]);
                uint32_t seen = 0xffffffffu;
                if (__builtin_expect(part, 0)) {
                    seen = 0;
#pragma unroll 1
                    for (int i = 0; i < NC; ++i) {
                        const int at = first + (i >> 1) * 8 + c0 + (i & 1);
                        if (at >= x.rq.n * a.G) continue;
                        const int tok = static_cast<int>(a.div_group.div(uint32_t(at)));
                        const uint32_t bits = sees32(a, x.rq.qs, tok, prefix, x.rq.len, tile * C::TN + k0);
                        seen |= ((bits & 1u) | (bits >> 6 & 4u)) << ((i >> 1) * 4 + (i & 1));
                    }
                    if constexpr (C::kWide)
#pragma unroll
                        for (int i = 0; i < C::SR / 2; ++i)
                            if (!(seen >> i & 1u)) s[i] = -INFINITY;
                }
                float most[2] = {-INFINITY, -INFINITY};  // of the thread's two rows, from the reference
#pragma unroll
                for (int i = 0; i < C::SR / 2; i += 2) {
                    const float2 y = from_reference(s, ref, qf, u, seen, i);
                    most[(i >> 1) & 1] = max3(most[(i >> 1) & 1], y.x, y.y);
                }
                bool moved = false;
                if (__builtin_expect(softmax_any(bar, it == 0 || sync->dead ||
                                                 fmaxf(most[0] + lu[0], most[1] + lu[1]) > C::kLag + C::kBias), 0)) {
                    if (softmax_any(bar, sync->dead)) return;
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        const int j = (i >> 1) * 4 + (i & 1);
                        const float f = C::kWide ? a.scale_log2 : qf[C::kWide ? 0 : i];
                        float top = C::kWide          ? s[j] * f
                                    : seen >> j & 1u ? s[j] * u[0] * f + lu[0]
                                                      : -INFINITY;
                        top = fmaxf(top, C::kWide              ? s[j + 2] * f
                                         : seen >> (j + 2) & 1u ? s[j + 2] * u[1] * f + lu[1]
                                                                : -INFINITY);
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        if (lane < 4) red[warp * C::SR + (i >> 1) * 8 + c0 - col0 + (i & 1)] = top;
                    }
                    softmax_sync(bar);
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        const int c = (i >> 1) * 8 + c0 + (i & 1);
                        const float* z = red + c - col0;
                        const float top = fmaxf(fmaxf(z[0], z[C::SR]), fmaxf(z[2 * C::SR], z[3 * C::SR]));
                        float f = 1.0f;
                        if (top - ref[i] > C::kLag + C::kBias || (it == 0 && top > -3.40282347e+38f)) {
                            const float to = top - C::kBias;
                            f = pow2(ref[i] - to);
                            ref[i] = to;
                            l[i] *= f;
                        }
                        if (tid < 4) sync->fac[c] = f;
                    }
                    softmax_sync(bar);
                    moved = it > 0;
                }
                // the weights' place is free, and O still, when the tile before is done
                if (n > 0) wait_product(n - 1);
                __syncwarp();
                if (__builtin_expect(moved, 0)) {
                    tmem_after();
                    shrink(lanes, col0);
                }
#pragma unroll
                for (int j = 0; j < J; j += 2) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // block j + k / 2, rows k % 2
                        const int i = (j + (k >> 1)) * 4 + (k & 1) * 2, c = (j + (k >> 1)) * 2;
                        float2 e = from_reference(s, ref, qf, u, seen, i);
                        e = make_float2(pow2(e.x), pow2(e.y));
                        const float2 sum = add2(make_float2(l[c], l[c + 1]), e);
                        l[c] = sum.x;
                        l[c + 1] = sum.y;
                        if constexpr (!C::kWide) {
                            e = mul2(e, make_float2(u[k & 1], u[k & 1]));
                            // (the scale need not be finite)
                            if (part && !(seen >> i & 1u)) e.x = 0.0f;
                            if (part && !(seen >> i & 2u)) e.y = 0.0f;
                        }
                        w[k] = pack2<C::BF16>(e.x, e.y);
                    }
                    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                                     p_at + j * 1024),
                                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                 : "memory");
                }
                if (__builtin_expect(part, 0) && C::STORE != ROPE_CACHE_INT8)
                    mend(n, max(prefix - tile * C::TN, 0), x.rq.len - tile * C::TN, run, group);
                to_async_proxy();
                tmem_before();
                bar_arrive(&sync->p_full);
            }
            // the run's results, when its last product is done
            wait_product(n - 1);
            if (softmax_any(bar, sync->dead)) return;
            tmem_after();
            finish(x, run, ref, l, lanes, group);
            tmem_before();
        }
    }

    // 16-bit rows of a chain: the first drafted row of the run's tiles whose value lane c is not
    // finite, and that value.  (Looked up once for all query rows: those of a chunk of 16000 tokens,
    // each looking at every row it sees, would take a second and more for a tile.)
    __device__ __noinline__ int first_not_finite(const RunAt x, int c, float* value) const {
        const int to = static_cast<int>(min(int64_t(x.rq.len), int64_t(x.t0 + x.count) * C::TN));
        for (int j = max(max(x.rq.len - x.rq.n, 0), x.t0 * C::TN); c < a.Dv && j < to; ++j) {
            const Row row = row_of(x, j);
            const uint32_t y = row.p ? __ldg(reinterpret_cast<const uint16_t*>(row.p) + c) : 0;
            if (!not_finite<C::STORE>(y)) continue;
            *value = value16<C::STORE>(y);
            return j;
        }
        return to;
    }

    __device__ __forceinline__ uint32_t pack_one(float y) const {
        return a.bf16 ? pack2<true>(y, 0.0f) : pack2<false>(y, 0.0f);
    }

    __device__ __forceinline__ void finish(const RunAt& x, uint32_t run, const float* ref, float* l,
                                           uint32_t lanes, int group) const {
        constexpr int NC = C::SR / 4;
        const int tid = int(threadIdx.x) & 127, lane = tid & 31, warp = tid >> 5, col0 = group * C::SR,
                  c0 = col0 + (lane & 3) * 2, bar = group + 1;
        float *red = sync->red + group * 4 * C::SR, *fac = sync->fac;
        const int first = x.m * C::ROWS, left = min(C::ROWS, x.rq.n * a.G - first);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i >> 1) * 8 + c0 + (i & 1);
#pragma unroll
            for (int d = 4; d < 32; d *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
            if (lane < 4) red[warp * C::SR + c - col0] = l[i];
            if (tid < 4) fac[c] = ref[i];
        }
        softmax_sync(bar);
        if (tid < C::SR) {
            const int row = col0 + tid;
            const float all = red[tid] + red[C::SR + tid] + red[2 * C::SR + tid] + red[3 * C::SR + tid];
            const float m = all == 0.0f ? -INFINITY : fac[row];
            fac[row] = x.slot >= 0 ? 1.0f : all == 0.0f ? 0.0f : 1.0f / all;
            if (x.slot >= 0) a.part_ml[x.slot * C::ROWS + row] = make_float2(m, all);
            else if (row < left) {
                const OutAt y = out_at(a, x.rq.qs, 0, first + row);
                if (y.lse) *y.lse = latent_lse(m, all);
            }
        }
        softmax_sync(bar);
        // where the rows of results lie: in the place of the sums, which have been read
        int64_t* rows = reinterpret_cast<int64_t*>(red);
        if (x.slot < 0) {
            if (tid < C::SR && col0 + tid < left) rows[tid] = out_at(a, x.rq.qs, 0, first + col0 + tid).out - a.out;
            softmax_sync(bar);
        }
        // Columns (query rows) of a lane by 16 or 32, turned over in a group's own part of the
        // weights' place.
        constexpr int W = C::SG == 2 || C::ROWS < 32 ? 16 : 32;
        const int tiles = value_tiles();
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            const int c = t * 128 + tid;
            const bool patch = C::kWide && sync->patch[run % 3][t] == run + 1;
            int spoilt = 0;
            float spoils = 0.0f;
            if constexpr (C::kWide)
                if (patch && !a.tree) spoilt = first_not_finite(x, c, &spoils);
#pragma unroll 1
            for (int r0 = col0; r0 < col0 + C::SR; r0 += W) {
                if (r0 >= left) break;
                float o[W];
                if constexpr (W == 32) tmem_ld32(o, lanes + t * C::ROWS + r0);
                else tmem_ld16(o, lanes + t * C::ROWS + r0);
                tmem_wait_ld();
                latent_here<W>(o);
                if (patch)
#pragma unroll 1
                    for (int r = 0; r < W && r0 + r < left; ++r) {
                        float add = 0.0f;
                        if (a.tree) {
                            if constexpr (C::kWide) add_not_finite<C::STORE, C::TN, 1>(a, x, first + r0 + r, c, &add);
                        } else if (int(a.div_group.div(uint32_t(first + r0 + r))) >= spoilt - (x.rq.len - x.rq.n)) {
                            add = spoils;
                        }
#pragma unroll
                        for (int k = 0; k < W; ++k) o[k] += k == r ? add : 0.0f;
                    }
                if (x.slot >= 0) {
                    float* to = a.part + (x.slot * C::ROWS + r0) * kLatentValues + c;
                    if (r0 + W <= left) {
#pragma unroll
                        for (int r = 0; r < W; ++r) to[r * kLatentValues] = o[r];
                    } else {
#pragma unroll
                        for (int r = 0; r < W; ++r)
                            if (r0 + r < left) to[r * kLatentValues] = o[r];
                    }
                    continue;
                }
                // turned over in the weights' place, rows of 128 lanes: 16 bytes a thread and store
                const uint32_t words = smem_addr(smem + C::P_AT) + group * 4096;
#pragma unroll
                for (int r = 0; r < W; ++r) {
                    const uint32_t y = pack_one(o[r] * fac[r0 + r]);
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(words + r * 256 + (((tid >> 3) ^ (r & 7)) << 4) +
                                                                 (tid & 7) * 2),
                                 "h"(static_cast<uint16_t>(y))
                                 : "memory");
                }
                softmax_sync(bar);
#pragma unroll
                for (int i = 0; i < W / 8; ++i) {
                    const int r = i * 8 + (tid >> 4), piece = tid & 15, at = t * 128 + piece * 8;
                    if (r0 + r < left && at < a.Dv) {
                        uint32_t w[4];
                        lds128(w, words + r * 256 + ((piece ^ (r & 7)) << 4));
                        *reinterpret_cast<uint4*>(a.out + rows[r0 - col0 + r] + at * 2) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                softmax_sync(bar);
            }
        }
        softmax_sync(bar);  // fac and red have been read
    }

    // The block's results, when one of its waits has given up: NaN in all of them, those
    // of the block's other runs too, and in its parts, whose joined results then are NaN.
    __device__ __noinline__ void give_up(const Place& place) const {
        const int tid = int(threadIdx.x);
        LatentWalk walk = latent_walk_from<C::ROWS, C::TN>(a, place);
        RunAt x;
        while (run_after(walk, x)) {
            const int first = x.m * C::ROWS, left = min(C::ROWS, x.rq.n * a.G - first);
            if (x.slot >= 0) {
                for (int r = tid; r < C::ROWS; r += kLatentThreads)
                    a.part_ml[x.slot * C::ROWS + r] = make_float2(-INFINITY, NAN);
                continue;
            }
            for (int i = tid; i < left * (a.Dv / 2); i += kLatentThreads) {
                const int row = i / (a.Dv / 2), c = i % (a.Dv / 2) * 2;
                const OutAt to = out_at(a, x.rq.qs, 0, first + row);
                *reinterpret_cast<uint32_t*>(to.out + c * 2) = 0x7fff7fffu;  // NaN of either type
                if (c == 0 && to.lse) *to.lse = NAN;
            }
        }
    }
};

// T: Latent, or what a test makes of it.
template <class T>
__global__ void __launch_bounds__(kLatentThreads, 1)
    rope_latent_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ LatentMaps maps) {
    using C = typename T::Cfg;
    extern __shared__ __align__(1024) char smem[];
    static_assert(C::SYNC_AT + int(sizeof(LatentSync)) + C::MORE <= C::kSmemMax, "shared memory");
    LatentSync* sync = reinterpret_cast<LatentSync*>(smem + C::SYNC_AT);
    const int warp = int(threadIdx.x) >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            for (int g = 0; g < 3; ++g) bar_init(&sync->full[i][g], C::BOXES ? 1 : C::TEAM);
            for (int g = 0; g < 2; ++g) bar_init(&sync->empty[i][g], 1);
            bar_init(&sync->s_full[i], 1);
            bar_init(&sync->s_free[i], 128 * C::SG);
        }
        bar_init(&sync->p_full, 128 * C::SG);
        bar_init(&sync->q_empty, 1);
        bar_init(&sync->done, 2);
        sync->dead = 0;
        for (int i = 0; i < 3; ++i) {
            for (int t = 0; t < 4; ++t) sync->patch[i][t] = 0;
            bar_init(&sync->run_full[i], 1);
            bar_init(&sync->q_full[i], C::HELPERS);
        }
        sync->taken = 0;
        sync->beat = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sync->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    after_predecessor();
    const Place place = find_place<C::ROWS, C::TN, kLatentThreads, true>(a, reinterpret_cast<int64_t*>(smem));
    tmem_before();
    __syncthreads();
    tmem_after();
    const T it{a, smem, sync, sync->tmem};
    if (warp < 4 || (C::SG == 2 && warp >= 8 && warp < 12)) {
        it.softmax(warp >> 3);
    } else if (warp == 4) {
        it.scores();
    } else if (warp == 5) {
        it.fetches(place, maps);
    } else if (warp < 14) {
        it.help(int(threadIdx.x) - (C::SG == 2 && warp >= 12 ? 320 : 192));
    } else {
        it.products();
    }
    if (warp == 4) it.all_done();
    tmem_before();
    __syncthreads();
    if (sync->dead) it.give_up(place);
    if (warp == 4) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sync->tmem));
    }
}

// Puts the parts of each split (request, row tile) together: out = sum_p O_p 2^(m_p - m) /
// sum_p l_p 2^(m_p - m).  A group cut by s block borders has s blocks here (times
// gridDim.y; of a pair of row tiles each has half of those), which share out its pieces of 128
// lanes of a row.  Up to 8 parts: a warp takes a piece, four lanes a thread, with its parts'
// loads in flight together; more: a block does, whose warps take the parts in turn and are
// added up in one order.
template <int ROWS>
__global__ void __launch_bounds__(kLatentJoinThreads) rope_latent_join_kernel(const __grid_constant__ TreeArgs a) {
    constexpr int WARPS = kLatentJoinThreads / 32;
    __shared__ float4 sums[WARPS][32];
    __shared__ float2 warp_ml[WARPS];
    after_predecessor();
    const int64_t b = int64_t(blockIdx.x) + 1;
    const TreeMeta w = a.meta[b];
    if (w.nt == 0) return;
    const int64_t from = w.u0 / w.chunk, to = (w.u0 + w.nt - 1) / w.chunk;
    const int parts = static_cast<int>(to - from + 1);
    const int qs = min(max(__ldg(a.q_start + w.r), 0), a.Tq);
    const int n = min(max(__ldg(a.q_start + w.r + 1), qs), a.Tq) - qs;
    // of a pair of row tiles this block joins one
    const int pair = a.share != a.G ? 1 : 0, odd = int(blockIdx.y) & pair, m = w.m + odd, shares = int(gridDim.y) >> pair;
    const int left = static_cast<int>(min(int64_t(ROWS), int64_t(n) * a.G - int64_t(m) * ROWS));
    const int lane = int(threadIdx.x) & 31, warp = int(threadIdx.x) >> 5, quarters = (a.Dv + 127) / 128;
    const int own = static_cast<int>(b - from - 1) * shares + (int(blockIdx.y) >> pair);
    const int all = (parts - 1) * shares;
    const int64_t before = int64_t(odd) * 2 * (gridDim.x + 1);  // parts of the pair's other
    // the part that begins the group has its block's second place
    auto slot = [&](int p) { return (before + (from + p) * 2 + (p == 0 ? 1 : 0)) * ROWS; };
    auto write = [&](int row, int c, float4 o, float top, float l) {
        const float norm = l == 0.0f ? 0.0f : 1.0f / l;
        const OutAt z = out_at(a, qs, 0, m * ROWS + row);
        if (c < a.Dv)
            *reinterpret_cast<uint2*>(z.out + c * 2) =
                a.bf16 ? make_uint2(pack2<true>(o.x * norm, o.y * norm), pack2<true>(o.z * norm, o.w * norm))
                       : make_uint2(pack2<false>(o.x * norm, o.y * norm), pack2<false>(o.z * norm, o.w * norm));
        if (c == 0 && z.lse) *z.lse = latent_lse(top, l);
    };
    // parts from p0 on, `step` apart
    auto gather = [&](int row, int c, int p0, int step, float4& o, float& top, float& l) {
        top = -INFINITY;
#pragma unroll 8
        for (int p = p0; p < parts; p += step) top = fmaxf(top, a.part_ml[slot(p) + row].x);
        const float base = top == -INFINITY ? 0.0f : top;
        o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        l = 0.0f;
#pragma unroll 8
        for (int p = p0; p < parts; p += step) {
            const float2 x = a.part_ml[slot(p) + row];
            const float4 y = *reinterpret_cast<const float4*>(a.part + (slot(p) + row) * kLatentValues + c);
            const float f = pow2(x.x - base);
            l += x.y * f;
            o.x += y.x * f;
            o.y += y.y * f;
            o.z += y.z * f;
            o.w += y.w * f;
        }
    };
    float4 o;
    float top, l;
    if (parts <= 8) {
        for (int i = own * WARPS + warp; i < left * quarters; i += all * WARPS) {
            const int row = i / quarters, c = (i - row * quarters) * 128 + lane * 4;
            gather(row, c, 0, 1, o, top, l);
            write(row, c, o, top, l);
        }
        return;
    }
    for (int i = own; i < left * quarters; i += all) {
        const int row = i / quarters, c = (i - row * quarters) * 128 + lane * 4;
        gather(row, c, warp, WARPS, o, top, l);
        sums[warp][lane] = o;
        if (lane == 0) warp_ml[warp] = make_float2(top, l);
        __syncthreads();
        if (warp == 0) {
            top = -INFINITY;
#pragma unroll
            for (int t = 0; t < WARPS; ++t) top = fmaxf(top, warp_ml[t].x);
            const float base = top == -INFINITY ? 0.0f : top;
            l = 0.0f;
            o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int t = 0; t < WARPS; ++t) {
                const float f = pow2(warp_ml[t].x - base);
                const float4 y = sums[t][lane];
                l += warp_ml[t].y * f;
                o.x += y.x * f;
                o.y += y.y * f;
                o.z += y.z * f;
                o.w += y.w * f;
            }
            write(row, c, o, top, l);
        }
        __syncthreads();
    }
}

template <class T>
TreeKernel latent_of() {
    using C = typename T::Cfg;
    return TreeKernel{reinterpret_cast<const void*>(&rope_latent_kernel<T>),
                      reinterpret_cast<const void*>(&rope_latent_join_kernel<C::ROWS>),
                      C::SYNC_AT + int(sizeof(LatentSync)) + C::MORE, kLatentThreads, C::TN, 0.0f, 0};
}

template <int STORE, int ROWS, bool BOXES>
TreeKernel latent_instance() {
    return latent_of<Latent<LatentCfg<STORE, ROWS, BOXES>>>();
}

template <int STORE>
TreeKernel latent_pick(const LatentPlan& p) {
    constexpr bool WIDE = STORE == ROPE_CACHE_BF16 || STORE == ROPE_CACHE_FP16;
    if constexpr (WIDE)
        if (p.boxes)
            return p.rows == 16   ? latent_instance<STORE, 16, true>()
                   : p.rows == 32 ? latent_instance<STORE, 32, true>()
                                  : latent_instance<STORE, 64, true>();
    return p.rows == 16   ? latent_instance<STORE, 16, false>()
           : p.rows == 32 ? latent_instance<STORE, 32, false>()
                          : latent_instance<STORE, 64, false>();
}

}  // namespace rope
