// rope_tree_common.cuh -- what the attention kernels share: the division of
// the work, the visibility of cache rows, the joining of parts.
//
// Units of work are (request, key head, row tile, cache tile), in that order (see kLead);
// every block takes an equal, contiguous run of them (one block per resident
// slot), so a long request is spread over many blocks and short ones share a
// block.  A block that holds a whole (request, head, row tile) writes the
// result; one that holds a part writes (O, m, l), and rope_tree_join_kernel
// puts the parts together.  Lengths are known on the device only: each block
// sums them itself (no plan pass, no host synchronisation).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <string.h>

#include "rope_tree.h"

namespace rope {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes from global to shared memory, zeros when !ok.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0)
                 : "memory");
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void lds128(uint32_t* r, uint32_t at) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ void lds64(uint32_t* r, uint32_t at) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// 2^x in one instruction (relative error 2^-22; 2^-inf = 0).
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t u;
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        memcpy(&u, &h, 4);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        memcpy(&u, &h, 4);
    }
    return u;
}

// The two codes in the low half (high half) of w as an fp16 pair, exactly.
//   fp8: a conversion instruction.  int8: the byte b ^ 128 = b + 128 under the
// exponent of 1024 is the fp16 number 1024 + 128 + b.
template <int STORE, bool HIGH>
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t w) {
    uint32_t r;
    if constexpr (STORE == ROPE_CACHE_FP8) {
        const uint16_t x = static_cast<uint16_t>(HIGH ? w >> 16 : w & 0xffffu);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
    } else {
        const uint32_t m = __byte_perm(w ^ 0x80808080u, 0x64646464u, HIGH ? 0x4342 : 0x4140);
        __half2 h;
        memcpy(&h, &m, 4);
        h = __hsub2(h, __half2half2(__ushort_as_half(0x6480)));  // 1152
        memcpy(&r, &h, 4);
    }
    return r;
}

// 16-bit values (the storage type's) that are not finite, and as numbers.
template <int STORE>
__device__ __forceinline__ bool not_finite(uint32_t x) {
    constexpr uint32_t e = STORE == ROPE_CACHE_BF16 ? 0x7f80u : 0x7c00u;
    return (x & e) == e;
}

template <int STORE>
__device__ __forceinline__ float value16(uint32_t x) {
    if constexpr (STORE == ROPE_CACHE_BF16) return __uint_as_float(x << 16);
    else return __half2float(__ushort_as_half(static_cast<unsigned short>(x)));
}

// Puts 0 in the place of e4m3 codes of NaN (0x7f and 0xff) in four words; not
// zero when there were any.
__device__ __forceinline__ uint32_t take_out_nan4(uint32_t* w) {
    uint32_t found = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t m = ((w[j] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // the top bit of such bytes
        w[j] &= ~((m >> 7) * 0xffu);
        found |= m;
    }
    return found;
}

// The power of two of a query row's largest |q| (its bit pattern `most`),
// kept within [2^-100, 2^100]; a row that is not finite needs none.
__device__ __forceinline__ float row_power(uint32_t most) {
    const uint32_t e = most & 0x7f800000u;
    return __uint_as_float(most >= 0x7f800000u
                               ? 0x3f800000u
                               : min(max(e, uint32_t(27) << 23), uint32_t(227) << 23));
}

// What a score is multiplied by in base 2, kept a normal number: 0 times the -inf
// of a row that is not seen, or infinity times a score of 0, would be NaN.
__device__ __forceinline__ float row_factor(float p, float scale_log2) {
    return fminf(fmaxf(p * scale_log2, 1.17549435e-38f), 3.40282347e+38f);
}

__device__ __forceinline__ float one_over_power(float p) {  // of a power of two
    return __uint_as_float(0x7f000000u - __float_as_uint(p));
}

// The power of two above x, within [2^-120, 2^120].
__device__ __forceinline__ float power_above(float x) {
    const uint32_t e = (__float_as_uint(x) & 0x7f800000u) + 0x00800000u;
    return __uint_as_float(min(max(e, uint32_t(7) << 23), uint32_t(247) << 23));
}

constexpr float kLeastPower = 7.5231638452626401e-37f;  // 2^-120

// Eight 16-bit values of q as fp32.
__device__ __forceinline__ void widen8(const uint4& x, bool bf16, float* f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (bf16) {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
            __half2 h;
            memcpy(&h, &w[j], 4);
            const float2 v = __half22float2(h);
            f[2 * j] = v.x;
            f[2 * j + 1] = v.y;
        }
    }
}

__device__ __forceinline__ uint32_t most_of(const float* f) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    return m;
}

__device__ __forceinline__ uint4 half8(const float* f, float by) {
    return make_uint4(pack2<false>(f[0] * by, f[1] * by), pack2<false>(f[2] * by, f[3] * by),
                      pack2<false>(f[4] * by, f[5] * by), pack2<false>(f[6] * by, f[7] * by));
}

// ------------------------------------------------------------------------
// the division of the work
// ------------------------------------------------------------------------

// Request r: groups (key heads x row tiles) of nt cache tiles (a request with no
// cache rows still has a tile, so that its results are written).
struct Request {
    int qs, n, len, mt, nt;
    int64_t groups;

    __device__ __forceinline__ int64_t units(int lead) const { return groups * (nt + lead); }
};

// A run of tiles costs its block its tiles and, once, what takes about as long as
// kLead of them: queries brought, the pipeline filled and drained, results written.
// So a group counts kLead units before those of its tiles, where a block has
// several tiles.  48 requests of 90 to 12000 fp8 rows, of which some blocks had
// four runs and some forty: 0 264 us, 2 252, 3 240, 4 232, 6 233; 12 requests of
// 6000 to 8200 bf16 rows: 112.9, 110.7, 110.6, 108.6, 112.2.
constexpr int kLead = 4;

// LATENT, here and below: row tiles hold a.share of the heads, and where groups count leads, the
// tiles that drafted rows fill (a request's last) count kMasked units more each, at their own
// place, so that a border between blocks may fall among them.
// Masks make such a tile that much slower.  With 0, 1, 2, 3 and 4: chunks of 200, 228 and 256 fp16
// tokens of 64 heads over 1031, 2565 and 4099 rows 459, 435, 408, 403 and 406 us; 1024 tokens of 4
// heads over 5120 rows 125, 114, 102, 103 and 116; of 16 heads over 8192 441, 434, 427, 434 and 442.
// (Counted before a group's first tile: 408, 153 and 485; 4096 tokens of one head over their own
// rows 310, where they take 153 here with any of these.)
// (The other kernels' groups are alike, and their walk has nothing of this: a lead worked out and
// carried for each request cost the first batch above 7 %.)
constexpr int kMasked = 3;

template <int TN, bool LATENT>
__device__ __forceinline__ int masked_tiles(const Request& q, int lead) {
    return LATENT && lead ? min(q.n / TN, q.nt) : 0;
}

template <int ROWS, int TN, bool LATENT>
__device__ __forceinline__ Request request(const TreeArgs& a, int r) {
    Request q;
    const int lo = min(max(__ldg(a.q_start + r), 0), a.Tq);
    const int hi = min(max(__ldg(a.q_start + r + 1), lo), a.Tq);
    q.qs = lo;
    q.n = hi - lo;
    q.len = min(max(__ldg(a.kv_len + r), 0), a.max_len);
    q.mt = static_cast<int>((int64_t(q.n) * (LATENT ? a.share : a.G) + ROWS - 1) / ROWS);
    q.nt = max(1, (q.len + TN - 1) / TN);
    q.groups = q.n == 0 ? 0 : int64_t(a.Hk) * q.mt;
    return q;
}

// A block's units, and the request that holds the first of them.
struct Place {
    int r, lead;
    int64_t base, start, end, chunk;  // base: units before request r
};

// Sum the requests' units, cut them into equal runs, and find this block's.
// All THREADS threads of the block take part; `scratch` holds THREADS / 16 + 2
// numbers of shared memory.
template <int ROWS, int TN, int THREADS, bool LATENT = false>
__device__ __forceinline__ Place find_place(const TreeArgs& a, int64_t* scratch) {
    constexpr int WARPS = THREADS / 32;
    int64_t* warp_sum = scratch;
    int64_t* warp_groups = scratch + WARPS;
    int64_t* found = scratch + 2 * WARPS;
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    int64_t mine = 0, groups = 0;
    for (int r = tid; r < a.R; r += THREADS) {
        const Request q = request<ROWS, TN, LATENT>(a, r);
        mine += q.units(0);
        groups += q.groups * (LATENT ? kLead + kMasked * masked_tiles<TN, LATENT>(q, kLead) : 1);
    }
#pragma unroll
    for (int d = 16; d; d /= 2) {
        mine += __shfl_xor_sync(0xffffffffu, mine, d);
        groups += __shfl_xor_sync(0xffffffffu, groups, d);
    }
    if (lane == 0) {
        warp_sum[warp] = mine;
        warp_groups[warp] = groups;
    }
    if (tid == 0) found[0] = a.R;
    __syncthreads();
    int64_t total = 0;
    groups = 0;
    for (int w = 0; w < WARPS; ++w) {
        total += warp_sum[w];
        groups += warp_groups[w];
    }
    Place p;
    p.lead = total >= int64_t(gridDim.x) * 8 ? kLead : 0;
    total += LATENT ? (p.lead ? groups : 0) : groups * p.lead;
    p.chunk = (total + gridDim.x - 1) / gridDim.x;
    if (p.chunk < 1) p.chunk = 1;
    p.start = int64_t(blockIdx.x) * p.chunk;
    p.end = min(p.start + p.chunk, total);
    p.r = a.R;
    p.base = 0;
    if (p.start >= total) return p;  // the same for the whole block
    int64_t before = 0;
    for (int r0 = 0; r0 < a.R; r0 += THREADS) {
        const int r = r0 + tid;
        int64_t u = 0;
        if (r < a.R) {
            const Request q = request<ROWS, TN, LATENT>(a, r);
            u = q.units(p.lead + kMasked * masked_tiles<TN, LATENT>(q, p.lead));
        }
        int64_t sum = u;  // inclusive over the warp
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t x = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += x;
        }
        __syncthreads();  // warp_sum has been read
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        int64_t base = before + sum - u;
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) base += warp_sum[w];
            before += warp_sum[w];
        }
        if (u > 0 && p.start >= base && p.start < base + u) {
            found[0] = r;
            found[1] = base;
        }
        if (before > p.start) break;  // the same for the whole block
    }
    __syncthreads();
    p.r = static_cast<int>(found[0]);
    p.base = found[1];
    return p;
}

// One run of a block: cache tiles [t0, t0 + count) of (request, head, row tile).
struct RunAt {
    Request rq;
    int r, h, m, t0, count;
    int64_t slot;  // where a part goes; -1: the run is whole
};

// A block's runs, one after the other; several warps may each walk them.  The
// group of the run is looked up once, by division, and then counted on.
struct Walk {
    Request q;
    int64_t u, end, g0;  // g0: the group's first unit (of its lead)
    int r, h, m, lead;
    bool first;
};

template <int ROWS, int TN>
__device__ __forceinline__ Walk walk_from(const TreeArgs& a, const Place& p) {
    Walk w{};
    w.u = p.start;
    w.end = p.end;
    w.lead = p.lead;
    w.first = true;
    if (w.u < w.end) {
        w.r = p.r;
        w.q = request<ROWS, TN, false>(a, w.r);
        const int each = w.q.nt + w.lead;
        const int64_t group = (w.u - p.base) / each;
        w.h = static_cast<int>(group / w.q.mt);
        w.m = static_cast<int>(group - int64_t(w.h) * w.q.mt);
        w.g0 = p.base + group * each;
    }
    return w;
}

template <int ROWS, int TN>
__device__ __forceinline__ bool next_run(const TreeArgs& a, Walk& w, RunAt& out) {
    if (w.u >= w.end) return false;
    if (w.u >= w.g0 + w.lead + w.q.nt) {  // the next group; there is one, as units are left
        w.g0 = w.u;
        if (++w.m == w.q.mt) {
            w.m = 0;
            if (++w.h == a.Hk) {
                w.h = 0;
                do {
                    if (++w.r >= a.R) return false;
                    w.q = request<ROWS, TN, false>(a, w.r);
                } while (w.q.groups == 0);
            }
        }
    }
    const int off = static_cast<int>(w.u - w.g0), before = max(w.lead - off, 0);  // units before the run's first tile
    if (w.end - w.u <= before) return false;
    RunAt x;
    x.rq = w.q;
    x.r = w.r;
    x.h = w.h;
    x.m = w.m;
    x.t0 = max(off - w.lead, 0);
    x.count = static_cast<int>(min(int64_t(w.q.nt - x.t0), w.end - w.u - before));
    x.slot = x.count == w.q.nt ? int64_t(-1) : int64_t(blockIdx.x) * 2 + (w.first ? 0 : 1);
    w.first = false;
    w.u += before + x.count;
    out = x;
    return true;
}

// The same for LATENT.  A tile belongs to the block that its first unit lies in, so a block may begin
// (or end) with units of a group and none of its tiles.  A part that begins its group has the
// block's second place, one that goes on has the first.
struct LatentWalk {
    Request q;
    int64_t u, end, g0;
    int r, m, lead;
    int masked;  // tiles of the request that count kMasked units more

    __device__ __forceinline__ int each() const { return lead + q.nt + kMasked * masked; }

    // The group's tiles whose units begin before unit p of it.
    __device__ __forceinline__ int tiles_before(int p) const {
        const int at = max(p - lead, 0), over = at - (q.nt - masked);
        return over <= 0 ? at : at - over + int(uint32_t(over + kMasked) / (1 + kMasked));
    }
};

template <int ROWS, int TN>
__device__ __forceinline__ LatentWalk latent_walk_from(const TreeArgs& a, const Place& p) {
    LatentWalk w{};
    w.u = p.start;
    w.end = p.end;
    w.lead = p.lead;
    if (w.u < w.end) {
        w.r = p.r;
        w.q = request<ROWS, TN, true>(a, w.r);
        w.masked = masked_tiles<TN, true>(w.q, w.lead);
        w.m = static_cast<int>((w.u - p.base) / w.each());
        w.g0 = p.base + int64_t(w.m) * w.each();
    }
    return w;
}

template <int ROWS, int TN>
__device__ __forceinline__ bool next_run(const TreeArgs& a, LatentWalk& w, RunAt& out) {
    RunAt x;
    int to;
    do {
        if (w.u >= w.end) return false;
        if (w.u >= w.g0 + w.each()) {  // the next group; there is one, as units are left
            w.g0 = w.u;
            if (++w.m == w.q.mt) {
                w.m = 0;
                do {
                    if (++w.r >= a.R) return false;
                    w.q = request<ROWS, TN, true>(a, w.r);
                } while (w.q.groups == 0);
                w.masked = masked_tiles<TN, true>(w.q, w.lead);
            }
        }
        const int off = static_cast<int>(w.u - w.g0), stop = static_cast<int>(min(w.end - w.g0, int64_t(w.each())));
        x.t0 = w.tiles_before(off);
        to = w.tiles_before(stop);
        w.u += stop - off;
    } while (to == x.t0);
    x.rq = w.q;
    x.r = w.r;
    x.h = 0;
    x.m = w.m;
    x.count = to - x.t0;
    x.slot = x.count == w.q.nt ? int64_t(-1) : int64_t(blockIdx.x) * 2 + (x.t0 == 0 ? 1 : 0);
    out = x;
    return true;
}

// What the join kernel needs to know of a block: the group that its first run
// belongs to, when that began in an earlier block.
__device__ __forceinline__ TreeMeta meta_of(const Place& p, const RunAt& x) {
    if (x.t0 == 0) return TreeMeta{0, p.chunk, 0, 0, 0, 0, p.lead};
    return TreeMeta{p.start - x.t0, p.chunk, x.r, x.h, x.m, x.rq.nt, p.lead};
}

// The same for LATENT, from the walk that has found the run: nt counts units, from the first tile's
// to the last's.
__device__ __forceinline__ TreeMeta meta_of(const Place& p, const LatentWalk& w, const RunAt& x) {
    if (x.t0 == 0) return TreeMeta{0, p.chunk, 0, 0, 0, 0, 0};
    return TreeMeta{w.g0 + w.lead, p.chunk, x.r, x.h, x.m, x.rq.nt + kMasked * max(w.masked - 1, 0), w.lead};
}

// Which of the 32 rows from j drafted token i of a request sees.
__device__ __forceinline__ uint32_t sees32(const TreeArgs& a, int qs, int i, int prefix, int len, int j) {
    const int cols = len - j;
    if (cols <= 0) return 0u;
    const uint32_t in = cols >= 32 ? 0xffffffffu : (1u << cols) - 1u;
    const int jj = j - prefix;
    if (jj <= -32) return in;
    if (!a.tree) {
        const int c = i - jj + 1;
        return c <= 0 ? 0u : c >= 32 ? in : in & ((1u << c) - 1u);
    }
    const int from = max(jj, 0), w = from >> 6, sh = from & 63;
    const unsigned long long* t =
        reinterpret_cast<const unsigned long long*>(a.tree) + int64_t(qs + i) * a.words;
    unsigned long long b = w < a.words ? __ldg(t + w) >> sh : 0ull;
    if (sh > 32 && w + 1 < a.words) b |= __ldg(t + w + 1) << (64 - sh);
    const uint32_t bits = static_cast<uint32_t>(b);
    return in & (jj < 0 ? (bits << -jj) | ((1u << -jj) - 1u) : bits);
}

// A drafted row's values that are not finite (8-bit: whose scale is not, or e4m3
// codes of NaN) are
// taken out of the product (a weight of 0 times infinity would reach the tokens that do not
// see the row) and added here to the tokens that do see it, which end up not
// finite in those columns whatever the weight: N columns from c of query row
// `at`, over the drafted rows of the run's tiles.
template <int STORE, int TN, int N>
__device__ __noinline__ void add_not_finite(const TreeArgs& a, const RunAt x, int at, int c, float* o) {
    const int i = static_cast<int>(a.div_group.div(uint32_t(at)));
    const int prefix = x.rq.len - x.rq.n;
    const int to = static_cast<int>(min(int64_t(x.rq.len), int64_t(x.t0 + x.count) * TN));
    for (int j = max(max(prefix, 0), x.t0 * TN); j < to; ++j) {
        if (!(sees32(a, x.rq.qs, i, prefix, x.rq.len, j) & 1u)) continue;
        uint32_t p, off;
        a.div_page.divmod(uint32_t(j), p, off);
        const int page = __ldg(a.table + int64_t(x.r) * a.table_stride + p);
        if (page < 0 || page >= a.pages) continue;
        if constexpr (STORE == ROPE_CACHE_BF16 || STORE == ROPE_CACHE_FP16) {
            const uint16_t* v = reinterpret_cast<const uint16_t*>(a.v + page * a.v_st[0] + int64_t(off) * a.v_st[1] +
                                                                  int64_t(x.h) * a.v_st[2]);
            for (int k = 0; k < N && c + k < a.Dv; ++k) {
                const uint32_t y = __ldg(v + c + k);
                if (not_finite<STORE>(y)) o[k] += value16<STORE>(y);
            }
        } else {
            // a scale that is not finite makes the whole row so
            const float y = __ldg(a.vs + page * a.vs_st[0] + int64_t(off) * a.vs_st[1] + int64_t(x.h) * a.vs_st[2]);
            const bool whole = !(fabsf(y) <= 3.4028234663852886e38f);
            const uint8_t* v = reinterpret_cast<const uint8_t*>(a.v + page * a.v_st[0] + int64_t(off) * a.v_st[1] +
                                                                int64_t(x.h) * a.v_st[2]);
            for (int k = 0; k < N && c + k < a.Dv; ++k)
                if (whole || (STORE == ROPE_CACHE_FP8 && (__ldg(v + c + k) & 0x7f) == 0x7f)) o[k] = NAN;
        }
    }
}

__device__ __forceinline__ void after_predecessor() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A result's place: row `at` of the request's n * G query rows of a key head.
struct OutAt {
    char* out;
    float* lse;  // null: not wanted
};

__device__ __forceinline__ OutAt out_at(const TreeArgs& a, int qs, int h, int at) {
    uint32_t tok, g;
    a.div_group.divmod(uint32_t(at), tok, g);
    const int64_t q = qs + int(tok), hq = h * a.G + int(g);
    return OutAt{a.out + q * a.o_st[0] + hq * a.o_st[1], a.lse ? a.lse + q * a.Hq + hq : nullptr};
}

__device__ __forceinline__ float lse_of(float top, float l, float bias) {
    return l == 0.0f ? -INFINITY : (top - bias + log2f(l)) * 0.69314718055994531f;
}

// Parts lie in blocks of RB rows (32, or the 16 of a narrow tile), columns one
// after the other with their rows side by side, so that a warp whose lanes are
// rows writes and reads 128 bytes at a time.
template <int ROWS, int DV>
struct PartAt {
    static constexpr int RB = ROWS < 32 ? ROWS : 32, BLOCKS = ROWS / RB;
    static __device__ __forceinline__ int64_t block(int64_t slot, int rb) { return (slot * BLOCKS + rb) * (DV * RB); }
};

// Puts the parts of each split (request, head, row tile) together: out =
// sum_p O_p 2^(m_p - m) / sum_p l_p 2^(m_p - m).  A group cut by s block
// borders has s blocks here (times gridDim.y), those whose run begins inside
// it, that share out its pieces.  The parts were written just before and come
// from L2, so what counts is the chain of latencies and how many run side by
// side.  Few parts: a warp takes a piece of 32 columns of a block of rows,
// alone, its lanes being rows (of two columns, when there are 16).  Many: a
// block takes a piece of 8 columns, its warps the parts in turn, joined
// through shared memory in the same order every time.  80 registers (three
// blocks an SM), so that a warp's loads of two parts are in flight together: 32 MB
// of parts (pairs of tiles cut by 151 borders) 11 us, where 64 registers took
// 14.6 and two blocks of 126 12.2.
template <int ROWS, int DV>
__global__ void __launch_bounds__(kJoinThreads, 3) rope_tree_join_kernel(const __grid_constant__ TreeArgs a,
                                                                      float bias) {
    using P = PartAt<ROWS, DV>;
    constexpr int WARPS = kJoinThreads / 32, RB = P::RB, CW = 8, WORDS = CW * RB;
    __shared__ float mine[WARPS][32][RB + 1];  // few: a warp's piece, a column after the other
    __shared__ float part[WARPS][WORDS];       // many: the warps' sums of a piece
    __shared__ float2 warp_ml[WARPS][RB];
    after_predecessor();
    const int64_t b = int64_t(blockIdx.x) + 1;
    const TreeMeta w = a.meta[b];
    if (w.nt == 0) return;
    const int64_t from = w.u0 / w.chunk, to = (w.u0 + w.nt - 1) / w.chunk;
    const int parts = static_cast<int>(to - from + 1);
    const int qs = min(max(__ldg(a.q_start + w.r), 0), a.Tq);
    const int n = min(max(__ldg(a.q_start + w.r + 1), qs), a.Tq) - qs;
    const int left = static_cast<int>(min(int64_t(ROWS), int64_t(n) * a.G - int64_t(w.m) * ROWS));
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, row = lane % RB;
    const int rbs = (left + RB - 1) / RB;
    const int own = static_cast<int>(b - from - 1) * int(gridDim.y) + int(blockIdx.y), all = (parts - 1) * int(gridDim.y);
    // part p of the group: block `from` holds it second unless the group
    // begins with the block's run (or before it, with the units of its lead);
    // the others hold it first
    const int64_t second = from * w.chunk < w.u0 - w.lead ? 1 : 0;
    auto slot = [&](int p) { return (from + p) * 2 + (p == 0 ? second : 0); };

    if (parts <= WARPS) {
        constexpr int E = RB;  // words of a lane
        for (int piece = own * WARPS + warp; piece < rbs * (DV / 32); piece += all * WARPS) {
            const int rb = piece / (DV / 32), c0 = piece % (DV / 32) * 32;
            const float2* ml = a.part_ml + rb * RB + row;
            float top = -INFINITY, l = 0.0f, o[E];
#pragma unroll 4
            for (int p = 0; p < parts; ++p) top = fmaxf(top, ml[slot(p) * ROWS].x);
            const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 2
            for (int p = 0; p < parts; ++p) {
                const float2 x = ml[slot(p) * ROWS];
                const float f = pow2(x.x - base);
                l += x.y * f;
                const float* src = a.part + P::block(slot(p), rb) + c0 * RB + lane;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] += src[e * 32] * f;
            }
            const float norm = l == 0.0f ? 0.0f : 1.0f / l;
            __syncwarp();
#pragma unroll
            for (int e = 0; e < E; ++e) mine[warp][(e * 32 + lane) / RB][row] = o[e] * norm;
            if (c0 == 0 && lane < RB && rb * RB + lane < left) {
                const OutAt y = out_at(a, qs, w.h, w.m * ROWS + rb * RB + lane);
                if (y.lse) *y.lse = lse_of(top, l, bias);
            }
            __syncwarp();
            // rows leave two columns a lane
            const int k = (lane & 15) * 2;
#pragma unroll 4
            for (int r = lane >> 4; r < RB; r += 2) {
                const int at = rb * RB + r;
                if (at < left && c0 + k < a.Dv) {
                    const float y = mine[warp][k][r], z = mine[warp][k + 1][r];
                    reinterpret_cast<uint32_t*>(out_at(a, qs, w.h, w.m * ROWS + at).out)[(c0 + k) / 2] =
                        a.bf16 ? pack2<true>(y, z) : pack2<false>(y, z);
                }
            }
        }
        return;
    }
    for (int piece = own; piece < rbs * (DV / CW); piece += all) {
        constexpr int E = WORDS / 32;
        const int rb = piece / (DV / CW), c0 = piece % (DV / CW) * CW;
        const float2* ml = a.part_ml + rb * RB + row;
        float top = -INFINITY, l = 0.0f, o[E];
#pragma unroll 4
        for (int p = warp; p < parts; p += WARPS) top = fmaxf(top, ml[slot(p) * ROWS].x);
        float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 4
        for (int p = warp; p < parts; p += WARPS) {
            const float2 x = ml[slot(p) * ROWS];
            const float f = pow2(x.x - base);
            l += x.y * f;
            const float* src = a.part + P::block(slot(p), rb) + c0 * RB + lane;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += src[e * 32] * f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) part[warp][e * 32 + lane] = o[e];
        if (lane < RB) warp_ml[warp][lane] = make_float2(top, l);
        __syncthreads();
        // a thread's word has the thread's row
        const int r = tid % RB;
        top = -INFINITY;
#pragma unroll
        for (int x = 0; x < WARPS; ++x) top = fmaxf(top, warp_ml[x][r].x);
        base = top == -INFINITY ? 0.0f : top;
        float y = 0.0f;
        l = 0.0f;
        if (tid < WORDS) {
#pragma unroll
            for (int x = 0; x < WARPS; ++x) {
                const float f = pow2(warp_ml[x][r].x - base);
                l += warp_ml[x][r].y * f;
                y += part[x][tid] * f;
            }
        }
        const int c = tid / RB, at = rb * RB + r;
        if (tid < WORDS && at < left) {
            const OutAt z = out_at(a, qs, w.h, w.m * ROWS + at);
            y *= l == 0.0f ? 0.0f : 1.0f / l;
            if (c0 + c < a.Dv)
                reinterpret_cast<uint16_t*>(z.out)[c0 + c] =
                    static_cast<uint16_t>(a.bf16 ? pack2<true>(y, 0.0f) : pack2<false>(y, 0.0f));
            if (c0 + c == 0 && z.lse) *z.lse = lse_of(top, l, bias);
        }
        __syncthreads();
    }
}

}  // namespace rope
