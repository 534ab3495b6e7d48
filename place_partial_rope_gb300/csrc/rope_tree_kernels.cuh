// rope_tree_kernels.cuh -- attention of drafted tokens over a paged cache.
//
// Mathematics.  The n drafted tokens of a request and the G query heads that
// share a key head are one matrix of n * G query rows (row = token * G +
// head of the group) against the same cache rows, so each cache row is read
// once for all of them.  Over tiles of TN cache rows, with s = q . k * scale
// in base 2, per query row:
//   m' = max(m, max_j s_j),  a = 2^(m - m'),  p_j = 2^(s_j - m'),
//   l = l a + sum_j p_j,     O = O a + sum_j p_j v_j,
// and out = O / l, lse = (m + log2 l) ln 2 at the end.  m starts at -inf; a
// row that has seen nothing keeps m = -inf, l = 0, O = 0.
//   8-bit caches: s_j gets the key's scale after the product, and p_j the
// value's before the rounding: p_j u_j / w with u_j the value's scale and w a
// power of two that is at least the largest u so far (O is multiplied by
// w_old / w_new, exactly, when it grows).  Codes become fp16 exactly, so the
// products are in fp16; q is brought to [-2, 2) by a power of two per row,
// which fp16 holds at bf16's precision whatever q's range, and which goes
// back into s.
//   fp16 products: p is scaled by 2^15 (kBias), so that weights down to 2^-39
// of the largest are kept, where fp16 alone would stop at 2^-24 and a long
// flat tail of small weights would vanish.
//   Rounding: p is rounded once to the product's 16-bit type; l sums the
// unrounded p; s, m, l and O are fp32.
//
// What bounds it.  A cache row costs (Dk + Dv) bytes per element byte and
// 2 n G (Dk + Dv) flops: HBM up to roughly 100 query rows at 16 bits.
//
// How.  Units of work are (request, key head, row tile, cache tile), laid out
// in that order; every block takes an equal, contiguous run of them (one
// block per resident slot), so a long request is spread over many blocks and
// short ones share a block.  A block that holds a whole (request, head, row
// tile) writes the result; one that holds a part writes (O, m, l), and the
// join kernel puts the parts together.  The lengths are known on the device
// only: each block sums them itself (no plan pass, no host synchronisation).
//   A block has four warps on a ring of STAGES tiles filled by cp.async, 16
// bytes a request, with the page numbers of a tile looked up one tile before
// its loads.  WM x WN warps: WM share out the query rows, WN the tile's
// cache rows; each of the WN keeps its own m, l, O, joined through shared
// memory when a run ends.  16-bit tiles go to the tensor cores by ldmatrix,
// 16-byte chunks swizzled by the row's low three bits.  8-bit tiles are read
// with 16-byte (8-byte) loads in an order of lanes that needs no shuffle:
// the sum over k may run in any order as long as q is permuted alike, and the
// columns of O may come in any order as long as the end puts them back; see
// key_frag and value_frag.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rope_tree.h"

namespace rope {

template <int STORE_, int DK_, int DV_, int MI_, int WM_, int WN_, int TN_, int STAGES_>
struct TreeCfg {
    static constexpr int STORE = STORE_, DK = DK_, DV = DV_, MI = MI_, WM = WM_, WN = WN_, TN = TN_,
                         STAGES = STAGES_;
    static constexpr bool kWide = STORE == ROPE_CACHE_BF16 || STORE == ROPE_CACHE_FP16;  // 16-bit codes
    static constexpr int ES = kWide ? 2 : 1;
    static constexpr int ROWS = 16 * MI * WM;   // query rows of a tile
    static constexpr int WROWS = 16 * MI;       // of a warp
    static constexpr int TW = TN / WN;          // cache rows of a tile per warp
    static constexpr int NT = TW / 8;           // 8-column tiles of s per warp
    static constexpr int NG = TW / 16;          // 16-row steps of p v per warp
    static constexpr int KS = DK / 16;          // 16-lane steps of q k
    static constexpr int ND = DV / 8;           // 8-column tiles of O
    static constexpr bool kQRegs = MI == 1 && DK <= 192;
    static constexpr int K_BYTES = TN * DK * ES, V_BYTES = TN * DV * ES;
    static constexpr int S_BYTES = kWide ? 0 : TN * 8;
    static constexpr int STAGE = K_BYTES + V_BYTES + S_BYTES;
    static constexpr int Q_BYTES = ROWS * DK * 2;
    static constexpr int QF_AT = Q_BYTES;
    static constexpr int INFO_AT = QF_AT + ROWS * 4;
    static constexpr int ML_AT = INFO_AT + STAGES * TN * 8;
    static constexpr int RING_AT = (ML_AT + WN * ROWS * 8 + 127) / 128 * 128;
    static constexpr int MERGE = WN * ROWS * DV * 4;
    static constexpr int SMEM = RING_AT + (STAGES * STAGE > MERGE ? STAGES * STAGE : MERGE);
    static constexpr float kBias = STORE == ROPE_CACHE_BF16 ? 0.0f : 15.0f;
    static_assert(32 * WM * WN == kTreeThreads, "four warps");
    static_assert(TN % (16 * WN) == 0 && TN <= kTreeThreads, "a tile's rows");
};

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

__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_t(uint32_t* r, uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
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

// c += a b, 16 x 16 times 16 x 8.
template <bool BF16>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    if constexpr (BF16) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    } else {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
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

// Where chunk ch (16 bytes) of row `row` of a tile lies.
template <class C>
__device__ __forceinline__ uint32_t key_at(int row, int ch) {
    if constexpr (C::kWide) return row * (C::DK * 2) + ((ch ^ (row & 7)) << 4);
    // 8-bit: a phase of eight lanes reads four chunks of two successive rows;
    // rows of 128 and 256 bytes need the two apart by half a line
    else if constexpr (C::DK % 128 == 0) return row * C::DK + ((ch ^ ((row & 1) << 2)) << 4);
    else return row * C::DK + (ch << 4);
}

template <class C>
__device__ __forceinline__ uint32_t value_at(int row, int ch) {
    if constexpr (C::kWide) return row * (C::DV * 2) + ((ch ^ (row & 7)) << 4);
    // 8-bit: a phase reads one or two chunks of rows 0, 2, 4, 6 (or 1, 3, 5, 7)
    else if constexpr (C::DV % 128 == 0) return row * C::DV + ((ch ^ (((row >> 1) & 3) << 1)) << 4);
    else {
        const int line = row >> 1, slot = (row & 1) * 4 + ch;
        return line * 128 + ((slot ^ ((line & 3) << 1)) << 4);
    }
}

// Units of request r: key heads x row tiles x cache tiles (a request with no
// cache rows still has a tile, so that its results are written).
struct Request {
    int qs, n, len, mt, nt;
    int64_t units;
};

template <class C>
__device__ __forceinline__ Request request(const TreeArgs& a, int r) {
    Request q;
    const int lo = min(max(__ldg(a.q_start + r), 0), a.Tq);
    const int hi = min(max(__ldg(a.q_start + r + 1), lo), a.Tq);
    q.qs = lo;
    q.n = hi - lo;
    q.len = min(max(__ldg(a.kv_len + r), 0), a.max_len);
    q.mt = static_cast<int>((int64_t(q.n) * a.G + C::ROWS - 1) / C::ROWS);
    q.nt = max(1, (q.len + C::TN - 1) / C::TN);
    q.units = q.n == 0 ? 0 : int64_t(a.Hk) * q.mt * q.nt;
    return q;
}

// Whether drafted token i (of the request) sees row j.
__device__ __forceinline__ bool sees(const TreeArgs& a, int qs, int i, int prefix, int len, int j) {
    if (j >= len) return false;
    const int jj = j - prefix;
    if (jj < 0) return true;
    if (!a.tree) return jj <= i;
    if (jj >= a.words * 64) return false;
    return (__ldg(reinterpret_cast<const long long*>(a.tree) + int64_t(qs + i) * a.words + (jj >> 6)) >>
            (jj & 63)) & 1;
}

// One run: cache tiles [t0, t0 + count) of (request, head h, row tile m).
template <class C>
struct Run {
    const TreeArgs& a;
    char* smem;
    Request rq;
    int r, h, m, t0, count;
    int64_t slot;  // where a part goes, -1: the run is whole

    static constexpr bool BF16 = C::STORE == ROPE_CACHE_BF16;

    // the page and offset of the tile's row `tid` (page -1: no such row)
    __device__ __forceinline__ int2 lookup(int tile) const {
        int2 at = make_int2(-1, 0);
        const int j = tile * C::TN + int(threadIdx.x);
        if (int(threadIdx.x) < C::TN && tile < t0 + count && j < rq.len) {
            uint32_t p, off;
            a.div_page.divmod(uint32_t(j), p, off);
            const int page = __ldg(a.table + int64_t(r) * a.table_stride + p);
            if (page >= 0 && page < a.pages) at = make_int2(page, int(off));
        }
        return at;
    }

    __device__ __forceinline__ void load_tile(int tile) const {
        if (tile < t0 + count) {
            const int2* info = reinterpret_cast<const int2*>(smem + C::INFO_AT) +
                               (tile - t0) % C::STAGES * C::TN;
            char* ring = smem + C::RING_AT + (tile - t0) % C::STAGES * C::STAGE;
            const uint32_t ks = smem_addr(ring), vs = ks + C::K_BYTES;
            constexpr int CK = C::DK * C::ES / 16, CV = C::DV * C::ES / 16;
            const char* kh = a.k + int64_t(h) * a.k_st[2];
            const char* vh = a.v + int64_t(h) * a.v_st[2];
#pragma unroll
            for (int i = 0; i < C::TN * CK / kTreeThreads; ++i) {
                const int at = int(threadIdx.x) + i * kTreeThreads, row = at / CK, ch = at % CK;
                const int2 w = info[row];
                const bool ok = w.x >= 0 && ch * 16 < a.Dk * C::ES;
                copy16(ks + key_at<C>(row, ch),
                       ok ? kh + w.x * a.k_st[0] + w.y * a.k_st[1] + ch * 16 : a.k, ok);
            }
#pragma unroll
            for (int i = 0; i < C::TN * CV / kTreeThreads; ++i) {
                const int at = int(threadIdx.x) + i * kTreeThreads, row = at / CV, ch = at % CV;
                const int2 w = info[row];
                const bool ok = w.x >= 0 && ch * 16 < a.Dv * C::ES;
                copy16(vs + value_at<C>(row, ch),
                       ok ? vh + w.x * a.v_st[0] + w.y * a.v_st[1] + ch * 16 : a.v, ok);
            }
            if constexpr (!C::kWide) {
                const int row = int(threadIdx.x);
                if (row < C::TN) {
                    const int2 w = info[row];
                    const bool ok = w.x >= 0;
                    const uint32_t at = vs + C::V_BYTES + row * 4;
                    copy4(at, ok ? a.ks + w.x * a.ks_st[0] + w.y * a.ks_st[1] + int64_t(h) * a.ks_st[2] : a.ks, ok);
                    copy4(at + C::TN * 4,
                          ok ? a.vs + w.x * a.vs_st[0] + w.y * a.vs_st[1] + int64_t(h) * a.vs_st[2] : a.vs, ok);
                }
            }
        }
        copies_commit();
    }

    // The row tile's queries into shared memory: 16-bit as they are (chunks
    // swizzled for ldmatrix), or fp16 in [-2, 2) with the power of two beside.
    __device__ __forceinline__ void stage_queries() const {
        constexpr int PER = kTreeThreads / C::ROWS;  // lanes of a row
        constexpr int N = C::DK / 8 / PER;           // chunks of a lane
        const int row = int(threadIdx.x) / PER, sub = int(threadIdx.x) % PER;
        const int at = m * C::ROWS + row;
        const bool there = at < rq.n * a.G;
        uint32_t tok = 0, g = 0;
        if (there) a.div_group.divmod(uint32_t(at), tok, g);
        const char* src = a.q + int64_t(rq.qs + int(tok)) * a.q_st[0] + int64_t(h * a.G + int(g)) * a.q_st[1];
        uint4 x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int ch = sub + i * PER;
            x[i] = there && ch * 8 < a.Dk ? __ldg(reinterpret_cast<const uint4*>(src) + ch)
                                          : make_uint4(0, 0, 0, 0);
        }
        if constexpr (C::kWide) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int ch = sub + i * PER;
                *reinterpret_cast<uint4*>(smem + row * C::DK * 2 + ((ch ^ (row & 7)) << 4)) = x[i];
            }
        } else {
            float f[N][8];
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (a.bf16) {
                        f[i][2 * j] = __uint_as_float(w[j] << 16);
                        f[i][2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                    } else {
                        __half2 hh;
                        memcpy(&hh, &w[j], 4);
                        const float2 ff = __half22float2(hh);
                        f[i][2 * j] = ff.x;
                        f[i][2 * j + 1] = ff.y;
                    }
                    most = max(most, max(__float_as_uint(f[i][2 * j]) & 0x7fffffffu,
                                         __float_as_uint(f[i][2 * j + 1]) & 0x7fffffffu));
                }
            }
#pragma unroll
            for (int d = PER / 2; d; d /= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
            // 2^e of the row's largest |q|, kept within [2^-100, 2^100]; a row
            // that is not finite needs none (its results are not either)
            uint32_t e = most & 0x7f800000u;
            e = most >= 0x7f800000u ? 0x3f800000u : min(max(e, uint32_t(27) << 23), uint32_t(227) << 23);
            const float down = __uint_as_float(0x7f000000u - e);
            if (sub == 0) reinterpret_cast<float*>(smem + C::QF_AT)[row] = __uint_as_float(e) * a.scale_log2;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int ch = sub + i * PER;
                uint4 y;
                y.x = pack2<false>(f[i][0] * down, f[i][1] * down);
                y.y = pack2<false>(f[i][2] * down, f[i][3] * down);
                y.z = pack2<false>(f[i][4] * down, f[i][5] * down);
                y.w = pack2<false>(f[i][6] * down, f[i][7] * down);
                *reinterpret_cast<uint4*>(smem + row * C::DK * 2 + ((ch ^ (row & 1)) << 4)) = y;
            }
        }
    }

    // The 16 x 16 fragment of q for step ks, or (8-bit) the four of steps
    // 4c .. 4c + 3: lane (g, t) takes lanes 64 c + 16 t .. + 15 of rows g and
    // g + 8, and step kk the four of them at 4 kk, as key_frag does.
    __device__ __forceinline__ void query_frag(uint32_t (*f)[4], int row0, int c) const {
        const int lane = int(threadIdx.x) & 31;
        if constexpr (C::kWide) {
            const int row = row0 + (lane & 15), ch = 2 * c + (lane >> 4);
            ldmatrix4(f[0], smem_addr(smem) + row * C::DK * 2 + ((ch ^ (row & 7)) << 4));
        } else {
            const int g = lane >> 2, t = lane & 3;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = row0 + g + 8 * half;
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int ch = 8 * c + 2 * t + i;
                    lds128(w + 4 * i, smem_addr(smem) + row * C::DK * 2 + ((ch ^ (row & 1)) << 4));
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    f[kk][half] = w[2 * kk];
                    f[kk][2 + half] = w[2 * kk + 1];
                }
            }
        }
    }

    __device__ __forceinline__ void go() {
        const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
        const int wm = warp % C::WM, wn = warp / C::WM;
        const int g = lane >> 2, t = lane & 3;
        const int row0 = wm * C::WROWS;
        int2* info = reinterpret_cast<int2*>(smem + C::INFO_AT);

        // page numbers of the first STAGES tiles, then the loads of all but one
        int2 first[C::STAGES];
#pragma unroll
        for (int i = 0; i < C::STAGES; ++i) first[i] = lookup(t0 + i);
        if (tid < C::TN) {
#pragma unroll
            for (int i = 0; i < C::STAGES; ++i) info[i * C::TN + tid] = first[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < C::STAGES - 1; ++i) load_tile(t0 + i);
        stage_queries();
        __syncthreads();

        constexpr int QSTEPS = C::kWide ? C::KS : C::KS / 4;  // calls of query_frag
        constexpr int QF = C::kWide ? 1 : 4;                  // fragments of a call
        uint32_t qreg[C::kQRegs ? C::KS : 1][4];
        if constexpr (C::kQRegs) {
#pragma unroll
            for (int c = 0; c < QSTEPS; ++c) query_frag(&qreg[c * QF], row0, c);
        }

        float mrow[C::MI][2], lrow[C::MI][2], qf[C::MI][2], O[C::MI][C::ND][4];
        int tok[C::MI][2];
        float vref = 7.5231638452626401e-37f;  // 2^-120: what w may not go below
#pragma unroll
        for (int i = 0; i < C::MI; ++i) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                mrow[i][b] = -INFINITY;
                lrow[i][b] = 0.0f;
                const int row = row0 + 16 * i + g + 8 * b;
                qf[i][b] = C::kWide ? a.scale_log2 : reinterpret_cast<const float*>(smem + C::QF_AT)[row];
                tok[i][b] = min(int(a.div_group.div(uint32_t(m * C::ROWS + row))), rq.n - 1);
            }
#pragma unroll
            for (int d = 0; d < C::ND; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[i][d][e] = 0.0f;
        }
        const int prefix = rq.len - rq.n;

        for (int it = 0; it < count; ++it) {
            const int tile = t0 + it;
            copies_wait<C::STAGES - 2>();
            __syncthreads();  // tile `it` is here, tile it - 1 is done with
            load_tile(tile + C::STAGES - 1);
            const int2 next = lookup(tile + C::STAGES);

            char* ring = smem + C::RING_AT + it % C::STAGES * C::STAGE;
            const uint32_t ks = smem_addr(ring), vs = ks + C::K_BYTES;
            const float* sk = reinterpret_cast<const float*>(ring + C::K_BYTES + C::V_BYTES);
            const float* sv = sk + C::TN;
            const int jw = wn * C::TW;  // this warp's first row of the tile

            // ---- s = q k
            float S[C::MI][C::NT][4];
#pragma unroll
            for (int i = 0; i < C::MI; ++i)
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[i][n][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < QSTEPS; ++c) {
                uint32_t qa[C::MI][QF][4];
#pragma unroll
                for (int i = 0; i < C::MI; ++i) {
                    if constexpr (C::kQRegs) {
#pragma unroll
                        for (int f = 0; f < QF; ++f)
#pragma unroll
                            for (int e = 0; e < 4; ++e) qa[i][f][e] = qreg[c * QF + f][e];
                    } else {
                        query_frag(qa[i], row0 + 16 * i, c);
                    }
                }
                if constexpr (C::kWide) {
#pragma unroll
                    for (int n = 0; n < C::NT; n += 2) {
                        const int row = jw + 8 * n + ((lane >> 4) << 3) + (lane & 7);
                        uint32_t b[4];
                        ldmatrix4(b, ks + key_at<C>(row, 2 * c + ((lane >> 3) & 1)));
#pragma unroll
                        for (int i = 0; i < C::MI; ++i) {
                            mma<BF16>(S[i][n], qa[i][0], b[0], b[1]);
                            mma<BF16>(S[i][n + 1], qa[i][0], b[2], b[3]);
                        }
                    }
                } else {
                    // lane (g, t): 16 codes of row g, four steps of the sum
#pragma unroll
                    for (int n = 0; n < C::NT; ++n) {
                        uint32_t w[4];
                        lds128(w, ks + key_at<C>(jw + 8 * n + g, 4 * c + t));
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            const uint32_t b0 = codes_to_half2<C::STORE, false>(w[f]);
                            const uint32_t b1 = codes_to_half2<C::STORE, true>(w[f]);
#pragma unroll
                            for (int i = 0; i < C::MI; ++i) mma<false>(S[i][n], qa[i][f], b0, b1);
                        }
                    }
                }
            }

            // ---- scales and the mask
            const int j0 = tile * C::TN + jw;
            const bool whole = tile * C::TN + C::TN <= prefix;  // context rows only
#pragma unroll
            for (int n = 0; n < C::NT; ++n) {
                float2 kk = make_float2(1.0f, 1.0f);
                if constexpr (!C::kWide) kk = *reinterpret_cast<const float2*>(sk + jw + 8 * n + 2 * t);
#pragma unroll
                for (int i = 0; i < C::MI; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float s = S[i][n][e] * qf[i][e >> 1];
                        if constexpr (!C::kWide) s *= (e & 1) ? kk.y : kk.x;
                        if (!whole && !sees(a, rq.qs, tok[i][e >> 1], prefix, rq.len, j0 + 8 * n + 2 * t + (e & 1)))
                            s = -INFINITY;
                        S[i][n][e] = s;
                    }
            }

            // ---- the running maximum; what is kept shrinks by 2^(m - m')
            float shrink[C::MI][2];
            bool moved = false;
#pragma unroll
            for (int i = 0; i < C::MI; ++i)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float top = -INFINITY;
#pragma unroll
                    for (int n = 0; n < C::NT; ++n) top = fmaxf(top, fmaxf(S[i][n][2 * b], S[i][n][2 * b + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    top = fmaxf(top, mrow[i][b]);
                    const float base = top == -INFINITY ? 0.0f : top;
                    shrink[i][b] = pow2(mrow[i][b] - base);
                    moved = moved || mrow[i][b] != top;
                    mrow[i][b] = top;
                    float sum = 0.0f;
#pragma unroll
                    for (int n = 0; n < C::NT; ++n)
#pragma unroll
                        for (int e = 2 * b; e < 2 * b + 2; ++e) {
                            S[i][n][e] = pow2(S[i][n][e] - (base - C::kBias));
                            sum += S[i][n][e];
                        }
                    lrow[i][b] = lrow[i][b] * shrink[i][b] + sum;
                }

            // ---- 8-bit: weights times the values' scales over their power of two
            if constexpr (!C::kWide) {
                float2 u[C::NT];
                float top = 0.0f;
#pragma unroll
                for (int n = 0; n < C::NT; ++n) {
                    u[n] = *reinterpret_cast<const float2*>(sv + jw + 8 * n + 2 * t);
                    top = fmaxf(top, fmaxf(u[n].x, u[n].y));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if (top > vref) {
                    // the power of two above `top`, at most 2^120
                    const float w = __uint_as_float(
                        min((__float_as_uint(top) & 0x7f800000u) + 0x00800000u, uint32_t(247) << 23));
                    const float f = vref / w;
                    vref = w;
                    moved = true;
#pragma unroll
                    for (int i = 0; i < C::MI; ++i)
#pragma unroll
                        for (int d = 0; d < C::ND; ++d)
#pragma unroll
                            for (int e = 0; e < 4; ++e) O[i][d][e] *= f;
                }
                const float back = __uint_as_float(0x7f000000u - __float_as_uint(vref));
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int i = 0; i < C::MI; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p = S[i][n][e];
                            // a row that is not seen adds nothing, whatever its scale
                            S[i][n][e] = p == 0.0f ? 0.0f : p * (((e & 1) ? u[n].y : u[n].x) * back);
                        }
            }

            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int i = 0; i < C::MI; ++i)
#pragma unroll
                    for (int d = 0; d < C::ND; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e) O[i][d][e] *= shrink[i][e >> 1];
            }

            if constexpr (C::kWide) {
                if (!whole) values_not_finite(vs, ring + C::K_BYTES, jw, S, O);
            }

            // ---- O += p v
#pragma unroll
            for (int n = 0; n < C::NG; ++n) {
                uint32_t p[C::MI][4];
#pragma unroll
                for (int i = 0; i < C::MI; ++i) {
                    p[i][0] = pack2<BF16>(S[i][2 * n][0], S[i][2 * n][1]);
                    p[i][1] = pack2<BF16>(S[i][2 * n][2], S[i][2 * n][3]);
                    p[i][2] = pack2<BF16>(S[i][2 * n + 1][0], S[i][2 * n + 1][1]);
                    p[i][3] = pack2<BF16>(S[i][2 * n + 1][2], S[i][2 * n + 1][3]);
                }
                const int jr = jw + 16 * n;
                if constexpr (C::kWide) {
#pragma unroll
                    for (int d = 0; d < C::ND; d += 2) {
                        uint32_t b[4];
                        ldmatrix4_t(b, vs + value_at<C>(jr + (lane & 15), d + (lane >> 4)));
#pragma unroll
                        for (int i = 0; i < C::MI; ++i) {
                            mma<BF16>(O[i][d], p[i], b[0], b[1]);
                            mma<BF16>(O[i][d + 1], p[i], b[2], b[3]);
                        }
                    }
                } else {
                    value_codes(vs, jr, p, O);
                }
            }
            if (tid < C::TN) info[it % C::STAGES * C::TN + tid] = next;
        }
        copies_wait<0>();
        finish(row0, wn, vref, mrow, lrow, O);
    }

    // 8-bit values.  Lane (g, t) needs, for column g of each 8-column tile, the
    // codes of rows 2t, 2t + 1, 2t + 8, 2t + 9.  It reads 16 (DV 64: 8)
    // successive columns of those four rows at once and takes its j-th column
    // as column g of tile j: tile j then holds columns DV / 8 * g + j (DV 256:
    // 128 p + 16 g + j), which finish() undoes.
    __device__ __forceinline__ void value_codes(uint32_t vs, int jr, const uint32_t (*p)[4],
                                                float (*O)[C::ND][4]) const {
        const int lane = int(threadIdx.x) & 31, g = lane >> 2, t = lane & 3;
        constexpr int W = C::DV == 64 ? 2 : 4;  // words of a read
#pragma unroll
        for (int pass = 0; pass < C::ND / (4 * W); ++pass) {
            uint32_t w[4][W];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int row = jr + 2 * t + (b & 1) + (b >> 1) * 8;
                if constexpr (W == 4) lds128(w[b], vs + value_at<C>(row, 8 * pass + g));
                else lds64(w[b], vs + value_at<C>(row, g >> 1) + (g & 1) * 8);
            }
#pragma unroll
            for (int x = 0; x < W; ++x) {
                const uint32_t lo0 = __byte_perm(w[0][x], w[1][x], 0x5140);
                const uint32_t hi0 = __byte_perm(w[0][x], w[1][x], 0x7362);
                const uint32_t lo1 = __byte_perm(w[2][x], w[3][x], 0x5140);
                const uint32_t hi1 = __byte_perm(w[2][x], w[3][x], 0x7362);
                const uint32_t b0[4] = {
                    codes_to_half2<C::STORE, false>(lo0), codes_to_half2<C::STORE, true>(lo0),
                    codes_to_half2<C::STORE, false>(hi0), codes_to_half2<C::STORE, true>(hi0)};
                const uint32_t b1[4] = {
                    codes_to_half2<C::STORE, false>(lo1), codes_to_half2<C::STORE, true>(lo1),
                    codes_to_half2<C::STORE, false>(hi1), codes_to_half2<C::STORE, true>(hi1)};
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int i = 0; i < C::MI; ++i)
                        mma<false>(O[i][pass * 4 * W + 4 * x + y], p[i], b0[y], b1[y]);
            }
        }
    }

    static __device__ __forceinline__ bool not_finite(uint32_t x) {  // a 16-bit value
        constexpr uint32_t e = C::STORE == ROPE_CACHE_BF16 ? 0x7f80u : 0x7c00u;
        return (x & e) == e;
    }

    static __device__ __forceinline__ float value16(uint32_t x) {
        if constexpr (C::STORE == ROPE_CACHE_BF16) return __uint_as_float(x << 16);
        else return __half2float(__ushort_as_half(static_cast<unsigned short>(x)));
    }

    // In a tile with rows that some tokens do not see, a value that is not
    // finite must not meet those tokens' weights of 0 in the product (0 * inf
    // is NaN).  Such values are rare: the block looks for one, and only then
    // adds their products by hand to the rows that do see them and puts zeros
    // in their place.
    __device__ __forceinline__ void values_not_finite(uint32_t vs, char* v, int jw, float (*S)[C::NT][4],
                                                      float (*O)[C::ND][4]) const {
        constexpr int N = C::TN * C::DV / 2;  // words of the tile
        uint32_t* w = reinterpret_cast<uint32_t*>(v);
        bool found = false;
        for (int i = int(threadIdx.x); i < N; i += kTreeThreads)
            found = found || not_finite(w[i] & 0xffffu) || not_finite(w[i] >> 16);
        if (!__syncthreads_or(found)) return;
        const int lane = int(threadIdx.x) & 31, t = lane & 3;
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
                const int row = jw + 8 * n + j, from = (lane & ~3) | (j >> 1);
#pragma unroll
                for (int i = 0; i < C::MI; ++i) {
                    float p[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float even = __shfl_sync(0xffffffffu, S[i][n][2 * b], from);
                        const float odd = __shfl_sync(0xffffffffu, S[i][n][2 * b + 1], from);
                        p[b] = j & 1 ? odd : even;
                    }
#pragma unroll
                    for (int d = 0; d < C::ND; ++d) {
                        const uint32_t x = w[(value_at<C>(row, d) >> 2) + t];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t y = e & 1 ? x >> 16 : x & 0xffffu;
                            if (not_finite(y) && p[e >> 1] != 0.0f) O[i][d][e] += p[e >> 1] * value16(y);
                        }
                    }
                }
            }
        }
        __syncthreads();
        for (int i = int(threadIdx.x); i < N; i += kTreeThreads) {
            const uint32_t x = w[i];
            w[i] = (not_finite(x & 0xffffu) ? 0u : x & 0xffffu) |
                   (not_finite(x >> 16) ? 0u : x & 0xffff0000u);
        }
        __syncthreads();
    }

    // The column of O[..][d][e & 1].
    static __device__ __forceinline__ int column(int d, int e, int t) {
        const int c = 2 * t + (e & 1);
        if constexpr (C::kWide) return 8 * d + c;
        else if constexpr (C::DV == 64) return 8 * c + d;
        else return d / 16 * 128 + 16 * c + d % 16;
    }

    // Join the WN warps' m, l, O of each row and write the result or the part.
    __device__ __forceinline__ void finish(int row0, int wn, float vref, float (*mrow)[2],
                                           float (*lrow)[2], float (*O)[C::ND][4]) const {
        const int tid = int(threadIdx.x), lane = tid & 31, g = lane >> 2, t = lane & 3;
        float2* ml = reinterpret_cast<float2*>(smem + C::ML_AT);
        float* part = reinterpret_cast<float*>(smem + C::RING_AT);
#pragma unroll
        for (int i = 0; i < C::MI; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float l = lrow[i][b];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                if (t == 0) ml[wn * C::ROWS + row0 + 16 * i + g + 8 * b] = make_float2(mrow[i][b], l);
            }
        __syncthreads();  // also: the ring is free
#pragma unroll
        for (int i = 0; i < C::MI; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int row = row0 + 16 * i + g + 8 * b;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < C::WN; ++w) top = fmaxf(top, ml[w * C::ROWS + row].x);
                float f = pow2(mrow[i][b] - (top == -INFINITY ? 0.0f : top));
                if constexpr (!C::kWide) f *= vref;
                float* to = part + (wn * C::ROWS + row) * C::DV;
#pragma unroll
                for (int d = 0; d < C::ND; ++d)
#pragma unroll
                    for (int e = 0; e < 2; ++e) to[column(d, e, t)] = O[i][d][2 * b + e] * f;
            }
        __syncthreads();
        constexpr int V = C::DV / 4;  // float4s of a row
        for (int i = tid; i < C::ROWS * V; i += kTreeThreads) {
            const int row = i / V, c = i % V * 4, at = m * C::ROWS + row;
            if (at >= rq.n * a.G) break;  // rows only grow with i
            float top = -INFINITY, l = 0.0f;
#pragma unroll
            for (int w = 0; w < C::WN; ++w) top = fmaxf(top, ml[w * C::ROWS + row].x);
            const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int w = 0; w < C::WN; ++w) {
                const float2 x = ml[w * C::ROWS + row];
                l += x.y * pow2(x.x - base);
            }
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < C::WN; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(part + (w * C::ROWS + row) * C::DV + c);
                o.x += x.x;
                o.y += x.y;
                o.z += x.z;
                o.w += x.w;
            }
            if (slot >= 0) {
                *reinterpret_cast<float4*>(a.part + (slot * C::ROWS + row) * C::DV + c) = o;
                if (c == 0) a.part_ml[slot * C::ROWS + row] = make_float2(top, l);
            } else {
                write_out(a, rq.qs, h, at, c, o, top, l, C::kBias);
            }
        }
        __syncthreads();  // before the next run reuses shared memory
    }

    // Four columns of one result.
    static __device__ __forceinline__ void write_out(const TreeArgs& a, int qs, int h, int at, int c,
                                                     float4 o, float top, float l, float bias) {
        uint32_t tok, g;
        a.div_group.divmod(uint32_t(at), tok, g);
        const int64_t q = qs + int(tok), hq = h * a.G + int(g);
        if (c == 0 && a.lse)
            a.lse[q * a.Hq + hq] = l == 0.0f ? -INFINITY : (top - bias + log2f(l)) * 0.69314718055994531f;
        if (c >= a.Dv) return;
        // a token that has seen no row gives zeros
        const float f = l == 0.0f ? 0.0f : 1.0f / l;
        uint2 y;
        if (a.bf16) y = make_uint2(pack2<true>(o.x * f, o.y * f), pack2<true>(o.z * f, o.w * f));
        else y = make_uint2(pack2<false>(o.x * f, o.y * f), pack2<false>(o.z * f, o.w * f));
        *reinterpret_cast<uint2*>(a.out + q * a.o_st[0] + hq * a.o_st[1] + c * 2) = y;
    }
};

// The request that holds a block's first unit, and the units before it.
struct Place {
    int r;
    int64_t base, start, end, chunk;
};

__device__ __forceinline__ void after_predecessor() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Sum the requests' units, cut them into equal runs, and find this block's.
template <class C>
__device__ __forceinline__ Place find_place(const TreeArgs& a) {
    __shared__ int64_t warp_sum[kTreeThreads / 32];
    __shared__ int64_t found_base;
    __shared__ int found_r;
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    int64_t mine = 0;
    for (int r = tid; r < a.R; r += kTreeThreads) mine += request<C>(a, r).units;
#pragma unroll
    for (int d = 16; d; d /= 2) mine += __shfl_xor_sync(0xffffffffu, mine, d);
    if (lane == 0) warp_sum[warp] = mine;
    if (tid == 0) found_r = a.R;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kTreeThreads / 32; ++w) total += warp_sum[w];
    Place p;
    p.chunk = (total + gridDim.x - 1) / gridDim.x;
    if (p.chunk < 1) p.chunk = 1;
    p.start = int64_t(blockIdx.x) * p.chunk;
    p.end = min(p.start + p.chunk, total);
    p.r = a.R;
    p.base = 0;
    if (p.start >= total) return p;  // the same for the whole block
    int64_t before = 0;
    for (int r0 = 0; r0 < a.R; r0 += kTreeThreads) {
        const int r = r0 + tid;
        const int64_t u = r < a.R ? request<C>(a, r).units : 0;
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
#pragma unroll
        for (int w = 0; w < kTreeThreads / 32; ++w) {
            if (w < warp) base += warp_sum[w];
            before += warp_sum[w];
        }
        if (u > 0 && p.start >= base && p.start < base + u) {
            found_r = r;
            found_base = base;
        }
        if (before > p.start) break;  // the same for the whole block
    }
    __syncthreads();
    p.r = found_r;
    p.base = found_base;
    return p;
}

template <class C>
__global__ void __launch_bounds__(kTreeThreads) rope_tree_kernel(const __grid_constant__ TreeArgs a) {
    extern __shared__ __align__(128) char smem[];
    after_predecessor();
    const Place p = find_place<C>(a);
    TreeMeta meta{0, p.chunk, 0, 0, 0, 0};
    int64_t u = p.start, base = p.base;
    int r = p.r;
    bool first = true;
    while (u < p.end && r < a.R) {
        const Request rq = request<C>(a, r);
        if (u >= base + rq.units) {
            base += rq.units;
            ++r;
            continue;
        }
        const int64_t per = int64_t(rq.mt) * rq.nt, at = u - base;
        const int h = static_cast<int>(at / per);
        const int rest = static_cast<int>(at - h * per);
        const int m = rest / rq.nt, t0 = rest - m * rq.nt;
        const int count = static_cast<int>(min(int64_t(rq.nt - t0), p.end - u));
        if (first && t0 > 0) meta = TreeMeta{u - t0, p.chunk, r, h, m, rq.nt};
        const bool all = count == rq.nt;
        Run<C> run{a, smem, rq, r, h, m, t0, count, all ? int64_t(-1) : int64_t(blockIdx.x) * 2 + (first ? 0 : 1)};
        run.go();
        first = false;
        u += count;
    }
    if (threadIdx.x == 0) a.meta[blockIdx.x] = meta;
}

// Puts the parts of each split (request, head, row tile) together: out =
// sum_p O_p 2^(m_p - m) / sum_p l_p 2^(m_p - m).  A group cut by s block
// borders has s blocks here (the ones whose run begins inside it) that share
// out its rows, so every block reads about as much as one of the main
// kernel's blocks wrote; blockIdx.y cuts that further.  Groups of few parts
// take a warp a row; of many, the whole block a row.  Bound by latency: the
// parts were written just before and come from L2.
template <int ROWS, int DV>
__global__ void __launch_bounds__(kJoinThreads) rope_tree_join_kernel(const __grid_constant__ TreeArgs a,
                                                                      float bias) {
    constexpr int WARPS = kJoinThreads / 32, V = DV / 32;  // columns of a lane
    __shared__ float sums[WARPS][DV];
    __shared__ float sum_l[WARPS];
    after_predecessor();
    const int64_t b = int64_t(blockIdx.x) + 1;
    const TreeMeta w = a.meta[b];
    if (w.nt == 0) return;
    const int64_t from = w.u0 / w.chunk, to = (w.u0 + w.nt - 1) / w.chunk;
    const int parts = static_cast<int>(to - from + 1), cuts = parts - 1;
    const int own = static_cast<int>(b - from - 1);
    const int qs = min(max(__ldg(a.q_start + w.r), 0), a.Tq);
    const int n = min(max(__ldg(a.q_start + w.r + 1), qs), a.Tq) - qs;
    const int left = min(ROWS, n * a.G - w.m * ROWS);  // rows of the tile
    const int lane = int(threadIdx.x) & 31, warp = int(threadIdx.x) >> 5;
    const bool alone = parts <= WARPS;  // a warp a row

    for (int k = int(blockIdx.y) + (alone ? warp * int(gridDim.y) : 0);; k += int(gridDim.y) * (alone ? WARPS : 1)) {
        const int row = own + cuts * k;
        if (row >= left) break;
        // part p of the group: block `from` holds it second unless the group
        // begins with the block's run; the others hold it first
        auto slot = [&](int p) { return (from + p) * 2 + (p == 0 && from * w.chunk != w.u0 ? 1 : 0); };
        float top = -INFINITY;
        for (int p = lane; p < parts; p += 32) top = fmaxf(top, a.part_ml[slot(p) * ROWS + row].x);
#pragma unroll
        for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == -INFINITY ? 0.0f : top;
        float o[V], l = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.0f;
#pragma unroll 4
        for (int p = alone ? 0 : warp; p < parts; p += alone ? 1 : WARPS) {
            const int64_t s = slot(p) * ROWS + row;
            const float2 x = a.part_ml[s];
            const float f = pow2(x.x - base);
            l += x.y * f;
            const float* src = a.part + s * DV + lane * V;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] += src[i] * f;
        }
        if (!alone) {
#pragma unroll
            for (int i = 0; i < V; ++i) sums[warp][lane * V + i] = o[i];
            if (lane == 0) sum_l[warp] = l;
            __syncthreads();
            l = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = 0.0f;
            if (warp == 0) {
                for (int x = 0; x < WARPS; ++x) {
                    l += sum_l[x];
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] += sums[x][lane * V + i];
                }
            }
            __syncthreads();
            if (warp != 0) continue;
        }
        uint32_t tok, g;
        a.div_group.divmod(uint32_t(w.m * ROWS + row), tok, g);
        const int64_t q = qs + int(tok), hq = w.h * a.G + int(g);
        if (lane == 0 && a.lse)
            a.lse[q * a.Hq + hq] = l == 0.0f ? -INFINITY : (top - bias + log2f(l)) * 0.69314718055994531f;
        const float f = l == 0.0f ? 0.0f : 1.0f / l;
        if (lane * V < a.Dv) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + q * a.o_st[0] + hq * a.o_st[1]) + lane * V / 2;
#pragma unroll
            for (int i = 0; i < V; i += 2)
                dst[i / 2] = a.bf16 ? pack2<true>(o[i] * f, o[i + 1] * f) : pack2<false>(o[i] * f, o[i + 1] * f);
        }
    }
}

// ------------------------------------------------------------------------
// kernel selection (instantiated in one .cu per storage type)
// ------------------------------------------------------------------------

struct TreeKernel {
    const void* main;
    const void* join;
    int smem;
    float bias;
};

template <int STORE, int DK, int DV, int MI, int WM, int WN>
TreeKernel tree_kernel() {
    // about 32 KB a stage and three stages, so that two blocks fit an SM
    constexpr bool wide = STORE == ROPE_CACHE_BF16 || STORE == ROPE_CACHE_FP16;
    constexpr int TN = wide ? 64 : (DK + DV > 256 ? 64 : 128);
    constexpr int per = TN * (DK + DV) * (wide ? 2 : 1);
    using C = TreeCfg<STORE, DK, DV, MI, WM, WN, TN, (per <= 32768 ? 3 : 2)>;
    return TreeKernel{reinterpret_cast<const void*>(&rope_tree_kernel<C>),
                      reinterpret_cast<const void*>(&rope_tree_join_kernel<C::ROWS, DV>), C::SMEM, C::kBias};
}

template <int STORE, int DK, int DV>
TreeKernel pick_tree_rows(const TreePlan& p) {
    if constexpr (DK <= 192) {
        if (p.rows == 64) return tree_kernel<STORE, DK, DV, 2, 2, 2>();
        if (p.rows == 32) return tree_kernel<STORE, DK, DV, 2, 1, 4>();
    }
    return tree_kernel<STORE, DK, DV, 1, 1, 4>();
}

template <int STORE>
TreeKernel pick_tree(const TreePlan& p) {
    if (p.dk == 64) return pick_tree_rows<STORE, 64, 64>(p);
    if (p.dk == 128) return pick_tree_rows<STORE, 128, 128>(p);
    if (p.dk == 192) return pick_tree_rows<STORE, 192, 128>(p);
    return pick_tree_rows<STORE, 256, 256>(p);
}

// defined in rope_tree_{bf16,fp16,fp8,int8}.cu
TreeKernel tree_kernel_bf16(const TreePlan& p);
TreeKernel tree_kernel_fp16(const TreePlan& p);
TreeKernel tree_kernel_fp8(const TreePlan& p);
TreeKernel tree_kernel_int8(const TreePlan& p);

}  // namespace rope
