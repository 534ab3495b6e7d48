// rope_tree_narrow.cuh -- attention of up to 16 query rows a key head (single
// tokens, small trees) over a paged cache, and of rows of 256 lanes.
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
// w_old / w_new, exactly, when it grows), over the rows that the query row sees:
// what the others hold has no effect on it.  Codes become fp16 exactly, so the
// products are in fp16; q is brought to [-2, 2) by a power of two per row,
// which fp16 holds at bf16's precision whatever q's range, and which goes
// back into s.
//   fp16 products: p is scaled by 2^15 (kBias), so that weights down to 2^-39
// of the largest are kept, where fp16 alone would stop at 2^-24 and a long
// flat tail of small weights would vanish.
//   Rounding: p is rounded once to the product's 16-bit type; l sums the
// unrounded p; s, m, l and O are fp32.
//
// What bounds it.  A cache row costs (Dk + Dv) times its element's bytes of
// HBM and 32 (Dk + Dv) flops on the 16-row tile: the bytes, four to eight
// times over.  So the legacy matrix instructions do (600 TFLOP/s measured on
// this card): their 16-row tile wastes less on a few rows than the 128 rows
// of tcgen05, and their results are in registers, where the softmax is.
//
// How.  A block has four warps on a ring of STAGES tiles filled by cp.async,
// 16 bytes a request, with the page numbers of a tile looked up one tile
// before its loads.  The warps share out the tile's cache rows; each keeps its
// own m, l, O, joined through shared memory when a run ends.  16-bit tiles go
// to the tensor cores by ldmatrix, 16-byte chunks swizzled by the row's low
// three bits.  8-bit tiles are read with 16-byte (8-byte) loads in an order of
// lanes that needs no shuffle: the sum over k may run in any order as long as
// q is permuted alike, and the columns of O may come in any order as long as
// the end puts them back; see query_frags and value_codes.
//   Measured (device, 8 query rows a key head, 8 key heads, 128 + 128 lanes): 32
// requests of 8000 fp8 rows 176 us, 3.0 TB/s (0.45 of the measured copy rate),
// what it issues bounding it; one request of 4097 bf16 rows and 2 key heads,
// 11 us, and 9 for the join (cold caches): latencies.
#pragma once
#include "rope_tree_common.cuh"

namespace rope {

template <int STORE_, int DK_, int DV_, int TN_, int STAGES_>
struct NarrowCfg {
    static constexpr int STORE = STORE_, DK = DK_, DV = DV_, TN = TN_, STAGES = STAGES_;
    static constexpr bool kWide = STORE == ROPE_CACHE_BF16 || STORE == ROPE_CACHE_FP16;  // 16-bit codes
    static constexpr int ES = kWide ? 2 : 1;
    static constexpr int ROWS = 16, WARPS = kNarrowThreads / 32;
    static constexpr int TW = TN / WARPS;  // cache rows of a tile per warp
    static constexpr int NT = TW / 8;      // 8-column tiles of s
    static constexpr int NG = TW / 16;     // 16-row steps of p v
    static constexpr int KS = DK / 16;     // 16-lane steps of q k
    static constexpr int ND = DV / 8;      // 8-column tiles of O
    static constexpr bool kQRegs = DK <= 192;
    static constexpr int K_BYTES = TN * DK * ES, V_BYTES = TN * DV * ES;
    static constexpr int STAGE = K_BYTES + V_BYTES + (kWide ? 0 : TN * 8);
    static constexpr int QF_AT = ROWS * DK * 2;
    static constexpr int INFO_AT = QF_AT + ROWS * 4;
    static constexpr int ML_AT = INFO_AT + STAGES * TN * 8;
    static constexpr int RING_AT = (ML_AT + WARPS * ROWS * 8 + 127) / 128 * 128;
    static constexpr int MERGE = WARPS * ROWS * DV * 4;
    static constexpr int SMEM = RING_AT + (STAGES * STAGE > MERGE ? STAGES * STAGE : MERGE);
    static constexpr float kBias = STORE == ROPE_CACHE_BF16 ? 0.0f : 15.0f;
    static_assert(TN % (16 * WARPS) == 0 && TN <= kNarrowThreads && TW <= 32, "a tile's rows");
};

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

// One run: cache tiles [t0, t0 + count) of (request, head h, row tile m).
template <class C>
struct Narrow {
    const TreeArgs& a;
    char* smem;
    RunAt x;

    static constexpr bool BF16 = C::STORE == ROPE_CACHE_BF16;
    static constexpr bool kMend = C::STORE != ROPE_CACHE_INT8;  // a value itself may be not finite

    // the page and offset of the tile's row `tid` (page -1: no such row)
    __device__ __forceinline__ int2 lookup(int tile) const {
        int2 at = make_int2(-1, 0);
        const int j = tile * C::TN + int(threadIdx.x);
        if (int(threadIdx.x) < C::TN && tile < x.t0 + x.count && j < x.rq.len) {
            uint32_t p, off;
            a.div_page.divmod(uint32_t(j), p, off);
            const int page = __ldg(a.table + int64_t(x.r) * a.table_stride + p);
            if (page >= 0 && page < a.pages) at = make_int2(page, int(off));
        }
        return at;
    }

    __device__ __forceinline__ void load_tile(int tile) const {
        if (tile < x.t0 + x.count) {
            const int st = (tile - x.t0) % C::STAGES;
            const int2* info = reinterpret_cast<const int2*>(smem + C::INFO_AT) + st * C::TN;
            const uint32_t ks = smem_addr(smem + C::RING_AT + st * C::STAGE), vs = ks + C::K_BYTES;
            constexpr int CK = C::DK * C::ES / 16, CV = C::DV * C::ES / 16;
            const char* kh = a.k + int64_t(x.h) * a.k_st[2];
            const char* vh = a.v + int64_t(x.h) * a.v_st[2];
#pragma unroll
            for (int i = 0; i < C::TN * CK / kNarrowThreads; ++i) {
                const int at = int(threadIdx.x) + i * kNarrowThreads, row = at / CK, ch = at % CK;
                const int2 w = info[row];
                const bool ok = w.x >= 0 && ch * 16 < a.Dk * C::ES;
                copy16(ks + key_at<C>(row, ch),
                       ok ? kh + w.x * a.k_st[0] + w.y * a.k_st[1] + ch * 16 : a.k, ok);
            }
#pragma unroll
            for (int i = 0; i < C::TN * CV / kNarrowThreads; ++i) {
                const int at = int(threadIdx.x) + i * kNarrowThreads, row = at / CV, ch = at % CV;
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
                    copy4(at, ok ? a.ks + w.x * a.ks_st[0] + w.y * a.ks_st[1] + int64_t(x.h) * a.ks_st[2] : a.ks, ok);
                    copy4(at + C::TN * 4,
                          ok ? a.vs + w.x * a.vs_st[0] + w.y * a.vs_st[1] + int64_t(x.h) * a.vs_st[2] : a.vs, ok);
                }
            }
        }
        copies_commit();
    }

    // The row tile's queries into shared memory: 16-bit as they are (chunks
    // swizzled for ldmatrix), or fp16 in [-2, 2) with the power of two beside.
    __device__ __forceinline__ void stage_queries() const {
        constexpr int PER = kNarrowThreads / C::ROWS;  // lanes of a row
        constexpr int N = C::DK / 8 / PER;             // chunks of a lane
        const int row = int(threadIdx.x) / PER, sub = int(threadIdx.x) % PER;
        const int at = x.m * C::ROWS + row;
        const bool there = at < x.rq.n * a.G;
        uint32_t tok = 0, g = 0;
        if (there) a.div_group.divmod(uint32_t(at), tok, g);
        const char* src = a.q + int64_t(x.rq.qs + int(tok)) * a.q_st[0] + int64_t(x.h * a.G + int(g)) * a.q_st[1];
        uint4 y[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int ch = sub + i * PER;
            y[i] = there && ch * 8 < a.Dk ? __ldg(reinterpret_cast<const uint4*>(src) + ch)
                                          : make_uint4(0, 0, 0, 0);
        }
        if constexpr (C::kWide) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int ch = sub + i * PER;
                *reinterpret_cast<uint4*>(smem + row * C::DK * 2 + ((ch ^ (row & 7)) << 4)) = y[i];
            }
        } else {
            float f[N][8];
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                widen8(y[i], a.bf16, f[i]);
                most = max(most, most_of(f[i]));
            }
#pragma unroll
            for (int d = PER / 2; d; d /= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
            const float p = row_power(most), down = one_over_power(p);
            if (sub == 0) reinterpret_cast<float*>(smem + C::QF_AT)[row] = row_factor(p, a.scale_log2);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int ch = sub + i * PER;
                *reinterpret_cast<uint4*>(smem + row * C::DK * 2 + ((ch ^ (row & 1)) << 4)) = half8(f[i], down);
            }
        }
    }

    // The 16 x 16 fragment of q for step c, or (8-bit) the four of steps
    // 4c .. 4c + 3: lane (g, t) takes lanes 64 c + 16 t .. + 15 of rows g and
    // g + 8, and step kk the four of them at 4 kk; keys are read alike.
    __device__ __forceinline__ void query_frags(uint32_t (*f)[4], int c) const {
        const int lane = int(threadIdx.x) & 31;
        if constexpr (C::kWide) {
            const int row = lane & 15, ch = 2 * c + (lane >> 4);
            ldmatrix4(f[0], smem_addr(smem) + row * C::DK * 2 + ((ch ^ (row & 7)) << 4));
        } else {
            const int g = lane >> 2, t = lane & 3;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = g + 8 * half;
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
        const int g = lane >> 2, t = lane & 3;
        int2* info = reinterpret_cast<int2*>(smem + C::INFO_AT);

        // page numbers of the first STAGES tiles, then the loads of all but one
        int2 first[C::STAGES];
#pragma unroll
        for (int i = 0; i < C::STAGES; ++i) first[i] = lookup(x.t0 + i);
        if (tid < C::TN) {
#pragma unroll
            for (int i = 0; i < C::STAGES; ++i) info[i * C::TN + tid] = first[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < C::STAGES - 1; ++i) load_tile(x.t0 + i);
        stage_queries();
        __syncthreads();

        constexpr int QSTEPS = C::kWide ? C::KS : C::KS / 4;  // calls of query_frags
        constexpr int QF = C::kWide ? 1 : 4;                  // fragments of a call
        uint32_t qreg[C::kQRegs ? C::KS : 1][4];
        if constexpr (C::kQRegs) {
#pragma unroll
            for (int c = 0; c < QSTEPS; ++c) query_frags(&qreg[c * QF], c);
        }

        float mrow[2], lrow[2], qf[2], O[C::ND][4];
        int tok[2];
        float vref[2] = {kLeastPower, kLeastPower};
        bool patch = false;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            mrow[b] = -INFINITY;
            lrow[b] = 0.0f;
            const int row = g + 8 * b;
            qf[b] = C::kWide ? a.scale_log2 : reinterpret_cast<const float*>(smem + C::QF_AT)[row];
            tok[b] = min(int(a.div_group.div(uint32_t(x.m * C::ROWS + row))), x.rq.n - 1);
        }
#pragma unroll
        for (int d = 0; d < C::ND; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[d][e] = 0.0f;
        const int prefix = x.rq.len - x.rq.n;

#pragma unroll 1
        for (int it = 0; it < x.count; ++it) {
            const int tile = x.t0 + it;
            copies_wait<C::STAGES - 2>();
            __syncthreads();  // tile `it` is here, tile it - 1 is done with
            load_tile(tile + C::STAGES - 1);
            const int2 next = lookup(tile + C::STAGES);

            char* ring = smem + C::RING_AT + it % C::STAGES * C::STAGE;
            const uint32_t ks = smem_addr(ring), vs = ks + C::K_BYTES;
            const float* sk = reinterpret_cast<const float*>(ring + C::K_BYTES + C::V_BYTES);
            const float* sv = sk + C::TN;
            const int jw = warp * C::TW;  // this warp's first row of the tile

            // ---- s = q k
            float S[C::NT][4];
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[n][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < QSTEPS; ++c) {
                uint32_t qa[QF][4];
                if constexpr (C::kQRegs) {
#pragma unroll
                    for (int f = 0; f < QF; ++f)
#pragma unroll
                        for (int e = 0; e < 4; ++e) qa[f][e] = qreg[c * QF + f][e];
                } else {
                    query_frags(qa, c);
                }
                if constexpr (C::kWide) {
#pragma unroll
                    for (int n = 0; n < C::NT; n += 2) {
                        const int row = jw + 8 * n + ((lane >> 4) << 3) + (lane & 7);
                        uint32_t b[4];
                        ldmatrix4(b, ks + key_at<C>(row, 2 * c + ((lane >> 3) & 1)));
                        mma<BF16>(S[n], qa[0], b[0], b[1]);
                        mma<BF16>(S[n + 1], qa[0], b[2], b[3]);
                    }
                } else {
                    // lane (g, t): 16 codes of row g, four steps of the sum
#pragma unroll
                    for (int n = 0; n < C::NT; ++n) {
                        uint32_t w[4];
                        lds128(w, ks + key_at<C>(jw + 8 * n + g, 4 * c + t));
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            mma<false>(S[n], qa[f], codes_to_half2<C::STORE, false>(w[f]),
                                       codes_to_half2<C::STORE, true>(w[f]));
                    }
                }
            }

            // ---- scales and the mask
            const bool whole = tile * C::TN + C::TN <= prefix;  // context rows only
            uint32_t sees[2] = {0xffffffffu, 0xffffffffu};
            if (!whole) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    sees[b] = sees32(a, x.rq.qs, tok[b], prefix, x.rq.len, tile * C::TN + jw);
            }
#pragma unroll
            for (int n = 0; n < C::NT; ++n) {
                float2 kk = make_float2(1.0f, 1.0f);
                if constexpr (!C::kWide) kk = *reinterpret_cast<const float2*>(sk + jw + 8 * n + 2 * t);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float s = S[n][e] * qf[e >> 1];
                    if constexpr (!C::kWide) s *= (e & 1) ? kk.y : kk.x;
                    S[n][e] = sees[e >> 1] >> (8 * n + 2 * t + (e & 1)) & 1u ? s : -INFINITY;
                }
            }

            // ---- the running maximum; what is kept shrinks by 2^(m - m')
            float shrink[2];
            bool moved = false;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float top = -INFINITY;
#pragma unroll
                for (int n = 0; n < C::NT; ++n) top = fmaxf(top, fmaxf(S[n][2 * b], S[n][2 * b + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                top = fmaxf(top, mrow[b]);
                const float base = top == -INFINITY ? 0.0f : top;
                shrink[b] = pow2(mrow[b] - base);
                moved = moved || mrow[b] != top;
                mrow[b] = top;
                float sum = 0.0f;
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int e = 2 * b; e < 2 * b + 2; ++e) {
                        S[n][e] = pow2(S[n][e] - (base - C::kBias));
                        sum += S[n][e];
                    }
                lrow[b] = lrow[b] * shrink[b] + sum;
            }

            // ---- 8-bit: weights times the values' scales over their power of two, which
            // is the query row's own: of the rows that it sees
            if constexpr (!C::kWide) {
                float2 u[C::NT];
                float top[2] = {0.0f, 0.0f};
#pragma unroll
                for (int n = 0; n < C::NT; ++n) u[n] = *reinterpret_cast<const float2*>(sv + jw + 8 * n + 2 * t);
                if (whole) {
#pragma unroll
                    for (int n = 0; n < C::NT; ++n) top[0] = fmaxf(top[0], fmaxf(u[n].x, u[n].y));
                    top[1] = top[0];
                } else {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int n = 0; n < C::NT; ++n) {
                            const uint32_t two = sees[b] >> (8 * n + 2 * t);
                            top[b] = fmaxf(top[b], fmaxf(two & 1u ? u[n].x : 0.0f, two & 2u ? u[n].y : 0.0f));
                        }
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    top[b] = fmaxf(top[b], __shfl_xor_sync(0xffffffffu, top[b], 1));
                    top[b] = fmaxf(top[b], __shfl_xor_sync(0xffffffffu, top[b], 2));
                    if (top[b] > vref[b]) {
                        const float w = power_above(top[b]), f = vref[b] / w;
                        vref[b] = w;
                        moved = true;
                        shrink[b] *= f;
                    }
                }
                const float back[2] = {one_over_power(vref[0]), one_over_power(vref[1])};
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = S[n][e];
                        // a row that is not seen adds nothing, whatever its scale
                        S[n][e] = p == 0.0f ? 0.0f : p * (((e & 1) ? u[n].y : u[n].x) * back[e >> 1]);
                    }
            }

            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int d = 0; d < C::ND; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[d][e] *= shrink[e >> 1];
            }

            if constexpr (kMend) {
                if (!whole && take_out_not_finite(ring + C::K_BYTES, prefix - tile * C::TN)) patch = true;
            }

            // ---- O += p v
#pragma unroll
            for (int n = 0; n < C::NG; ++n) {
                const uint32_t p[4] = {
                    pack2<BF16>(S[2 * n][0], S[2 * n][1]), pack2<BF16>(S[2 * n][2], S[2 * n][3]),
                    pack2<BF16>(S[2 * n + 1][0], S[2 * n + 1][1]), pack2<BF16>(S[2 * n + 1][2], S[2 * n + 1][3])};
                const int jr = jw + 16 * n;
                if constexpr (C::kWide) {
#pragma unroll
                    for (int d = 0; d < C::ND; d += 2) {
                        uint32_t b[4];
                        ldmatrix4_t(b, vs + value_at<C>(jr + (lane & 15), d + (lane >> 4)));
                        mma<BF16>(O[d], p, b[0], b[1]);
                        mma<BF16>(O[d + 1], p, b[2], b[3]);
                    }
                } else {
                    value_codes(vs, jr, p, O);
                }
            }
            if (tid < C::TN) info[it % C::STAGES * C::TN + tid] = next;
        }
        copies_wait<0>();
        finish(warp, vref, mrow, lrow, O, patch);
    }

    // 8-bit values.  Lane (g, t) needs, for column g of each 8-column tile, the
    // codes of rows 2t, 2t + 1, 2t + 8, 2t + 9.  It reads 16 (DV 64: 8)
    // successive columns of those four rows at once and takes its j-th column
    // as column g of tile j: tile j then holds columns DV / 8 * g + j (DV 256:
    // 128 p + 16 g + j), which finish() undoes.
    __device__ __forceinline__ void value_codes(uint32_t vs, int jr, const uint32_t* p, float (*O)[4]) const {
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
            for (int y = 0; y < W; ++y) {
                const uint32_t lo0 = __byte_perm(w[0][y], w[1][y], 0x5140);
                const uint32_t hi0 = __byte_perm(w[0][y], w[1][y], 0x7362);
                const uint32_t lo1 = __byte_perm(w[2][y], w[3][y], 0x5140);
                const uint32_t hi1 = __byte_perm(w[2][y], w[3][y], 0x7362);
                float(*o)[4] = &O[pass * 4 * W + 4 * y];
                mma<false>(o[0], p, codes_to_half2<C::STORE, false>(lo0), codes_to_half2<C::STORE, false>(lo1));
                mma<false>(o[1], p, codes_to_half2<C::STORE, true>(lo0), codes_to_half2<C::STORE, true>(lo1));
                mma<false>(o[2], p, codes_to_half2<C::STORE, false>(hi0), codes_to_half2<C::STORE, false>(hi1));
                mma<false>(o[3], p, codes_to_half2<C::STORE, true>(hi0), codes_to_half2<C::STORE, true>(hi1));
            }
        }
    }

    // Puts zeros in the place of values that are not finite (e4m3: of codes of NaN)
    // in the tile's rows from `from` on; whether there were any (see add_not_finite).
    static __device__ __noinline__ bool take_out_not_finite(char* v, int from) {
        bool found = false;
        if constexpr (C::kWide) {
            uint32_t* w = reinterpret_cast<uint32_t*>(v);
            for (int i = max(from, 0) * (C::DV / 2) + int(threadIdx.x); i < C::TN * C::DV / 2; i += kNarrowThreads) {
                const uint32_t y = w[i];
                const bool lo = not_finite<C::STORE>(y & 0xffffu), hi = not_finite<C::STORE>(y >> 16);
                if (lo || hi) {
                    found = true;
                    w[i] = (lo ? 0u : y & 0xffffu) | (hi ? 0u : y & 0xffff0000u);
                }
            }
        } else {
            constexpr int CH = C::DV / 16;
            for (int i = max(from, 0) * CH + int(threadIdx.x); i < C::TN * CH; i += kNarrowThreads) {
                const uint32_t at = smem_addr(v) + value_at<C>(i / CH, i % CH);
                uint32_t w[4];
                lds128(w, at);
                if (take_out_nan4(w)) {
                    found = true;
                    sts128(at, w[0], w[1], w[2], w[3]);
                }
            }
        }
        return __syncthreads_or(found);
    }

    // The column of O[d][e & 1].
    static __device__ __forceinline__ int column(int d, int e, int t) {
        const int c = 2 * t + (e & 1);
        if constexpr (C::kWide) return 8 * d + c;
        else if constexpr (C::DV == 64) return 8 * c + d;
        else return d / 16 * 128 + 16 * c + d % 16;
    }

    // Join the warps' m, l, O of each row and write the result or the part.
    __device__ __forceinline__ void finish(int warp, const float* vref, const float* mrow, const float* lrow,
                                           float (*O)[4], bool patch) const {
        const int tid = int(threadIdx.x), lane = tid & 31, g = lane >> 2, t = lane & 3;
        float2* ml = reinterpret_cast<float2*>(smem + C::ML_AT);
        float* part = reinterpret_cast<float*>(smem + C::RING_AT);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float l = lrow[b];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if (t == 0) ml[warp * C::ROWS + g + 8 * b] = make_float2(mrow[b], l);
        }
        __syncthreads();  // also: the ring is free
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int row = g + 8 * b;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < C::WARPS; ++w) top = fmaxf(top, ml[w * C::ROWS + row].x);
            float f = pow2(mrow[b] - (top == -INFINITY ? 0.0f : top));
            if constexpr (!C::kWide) f *= vref[b];
            float* to = part + warp * (C::ROWS * C::DV) + row;
#pragma unroll
            for (int d = 0; d < C::ND; ++d)
#pragma unroll
                for (int e = 0; e < 2; ++e) to[column(d, e, t) * C::ROWS] = O[d][2 * b + e] * f;
        }
        __syncthreads();
        // four columns of a row a thread, rows side by side
        for (int i = tid; i < C::ROWS * (C::DV / 4); i += kNarrowThreads) {
            const int row = i % C::ROWS, c = i / C::ROWS * 4, at = x.m * C::ROWS + row;
            if (at >= x.rq.n * a.G) continue;
            float top = -INFINITY, l = 0.0f;
#pragma unroll
            for (int w = 0; w < C::WARPS; ++w) top = fmaxf(top, ml[w * C::ROWS + row].x);
            const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int w = 0; w < C::WARPS; ++w) {
                const float2 y = ml[w * C::ROWS + row];
                l += y.y * pow2(y.x - base);
            }
            float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < C::WARPS; ++w)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] += part[w * (C::ROWS * C::DV) + (c + k) * C::ROWS + row];
            if constexpr (kMend) {
                if (patch) add_not_finite<C::STORE, C::TN, 4>(a, x, at, c, o);
            }
            if (x.slot >= 0) {
                float* to = a.part + PartAt<C::ROWS, C::DV>::block(x.slot, 0) + c * C::ROWS + row;
#pragma unroll
                for (int k = 0; k < 4; ++k) to[k * C::ROWS] = o[k];
                if (c == 0) a.part_ml[x.slot * C::ROWS + row] = make_float2(top, l);
            } else {
                const OutAt to = out_at(a, x.rq.qs, x.h, at);
                if (c == 0 && to.lse) *to.lse = lse_of(top, l, C::kBias);
                if (c < a.Dv) {
                    // a token that has seen no row gives zeros
                    const float f = l == 0.0f ? 0.0f : 1.0f / l;
                    uint2 y;
                    if (a.bf16) y = make_uint2(pack2<true>(o[0] * f, o[1] * f), pack2<true>(o[2] * f, o[3] * f));
                    else y = make_uint2(pack2<false>(o[0] * f, o[1] * f), pack2<false>(o[2] * f, o[3] * f));
                    *reinterpret_cast<uint2*>(to.out + c * 2) = y;
                }
            }
        }
        __syncthreads();  // before the next run reuses shared memory
    }
};

template <class C>
__global__ void __launch_bounds__(kNarrowThreads) rope_tree_narrow_kernel(const __grid_constant__ TreeArgs a) {
    extern __shared__ __align__(128) char smem[];
    after_predecessor();
    const Place p = find_place<C::ROWS, C::TN, kNarrowThreads>(a, reinterpret_cast<int64_t*>(smem));
    Walk walk = walk_from<C::ROWS, C::TN>(a, p);
    TreeMeta meta{0, p.chunk, 0, 0, 0, 0, 0};
    RunAt step;
    bool first = true;
    __syncthreads();  // the place's scratch is done with
    while (next_run<C::ROWS, C::TN>(a, walk, step)) {
        const RunAt x = step;
        if (first) meta = meta_of(p, x);
        first = false;
        Narrow<C>{a, smem, x}.go();
    }
    if (threadIdx.x == 0) a.meta[blockIdx.x] = meta;
}

template <int STORE, int DK, int DV>
TreeKernel narrow_kernel() {
    // about 32 KB a stage and three stages, so that two blocks fit an SM
    constexpr bool wide = STORE == ROPE_CACHE_BF16 || STORE == ROPE_CACHE_FP16;
    constexpr int TN = wide ? 64 : (DK + DV > 256 ? 64 : 128);
    constexpr int per = TN * (DK + DV) * (wide ? 2 : 1);
    using C = NarrowCfg<STORE, DK, DV, TN, (per <= 32768 ? 3 : 2)>;
    return TreeKernel{reinterpret_cast<const void*>(&rope_tree_narrow_kernel<C>),
                      reinterpret_cast<const void*>(&rope_tree_join_kernel<C::ROWS, DV>), C::SMEM,
                      kNarrowThreads, C::TN, C::kBias, 0};
}

}  // namespace rope
