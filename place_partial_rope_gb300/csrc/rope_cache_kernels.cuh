// rope_cache_kernels.cuh -- writing a paged cache of rotated keys and of
// values, and reading it back.
//
// Mathematics, per row x (one token, one head, keys or values) in fp32:
//   write  keys: lanes [start, end) turn as in rope_partial_kernel (each
//          product and sum one rounding); then, for an 8-bit cache,
//          m = max(max_i |x_i|, 2^-100), scale = m / top,
//          code_i = rn(x_i * (top / m)), top = 448 (e4m3) or 127;
//          for a 16-bit cache value_i = rn(x_i).
//   read   x_i = rn(code_i * scale).
// The maximum is taken over the bit patterns of |x|, which order like the
// numbers with infinity and NaN above them, so one integer maximum also tells
// whether a row is finite; one that is not stores a NaN scale and zero codes.
// One reciprocal a row and a product a lane, instead of a division a lane:
// the division would make the kernel issue-bound (about 10 instructions a
// lane against 4).
//
// What bounds it: HBM, one pass over the rows.  A row is spread over 8 lanes
// (32 for rows of more than 256) in whole 8-element accesses, kept in registers
// between the maximum and the rounding, so it is read once.  Eight lanes, where
// one access a lane would take 16 or 24: a lane then has 2 or 3 accesses of its
// row in flight, idles in no row length that 64 divides, and the maximum takes 3
// shuffles.  Rows of a token's keys and values follow each other in the work
// index, so that a warp's accesses lie side by side.  (A group of lanes with two
// or four heads of a token, their loads issued together and one slot looked up,
// was slower: reading 65536 rows of 8 heads of 128 fp8 codes took 97 and 148 us
// against 77 with one.)  Rows that are not aligned for 8-element accesses go one
// element an access (V 1).  8-bit rows are read by four lanes in accesses of 16
// codes: 69 us against 75 in the case above; writing them so took 160 us for
// 16411 tokens (and reading back) of 16 heads of 192 + 128, against 117.
// Measured: those 16411 bf16 tokens into int8, 70 us for 254 MB, 0.54 of the
// measured copy rate: a row is a chain of loads, rotation, maximum and rounding, of
// which 64 registers a thread let half the warps be in flight (2.4 of 4 instructions a
// cycle, 5.4 long-scoreboard stalls an issue).  Back,
// 46 us, 0.84; the 65536 rows above 69 us (407 MB), 0.89.
#pragma once
#include <cuda_fp8.h>

#include "rope_cache.h"
#include "rope_kernels.cuh"

namespace rope {

template <int STORE>
struct Store;

template <>
struct Store<ROPE_CACHE_BF16> {
    static constexpr int kBytes = 2;
    static constexpr float kTop = 0.0f;
    static __device__ __forceinline__ uint32_t put(float v) { return Elem<__nv_bfloat16>::put(v); }
    static __device__ __forceinline__ float get(uint32_t w) { return __uint_as_float((w & 0xffffu) << 16); }
};

template <>
struct Store<ROPE_CACHE_FP16> {
    static constexpr int kBytes = 2;
    static constexpr float kTop = 0.0f;
    static __device__ __forceinline__ uint32_t put(float v) { return Elem<__half>::put(v); }
    static __device__ __forceinline__ float get(uint32_t w) { return Elem<__half>::get(w); }
};

template <>
struct Store<ROPE_CACHE_FP8> {
    static constexpr int kBytes = 1;
    static constexpr float kTop = 448.0f;
    static __device__ __forceinline__ uint32_t put(float v) {
        return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
    }
    static __device__ __forceinline__ float get(uint32_t w) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(w & 0xffu), __NV_E4M3);
        return __half2float(__half(h));
    }
};

template <>
struct Store<ROPE_CACHE_INT8> {
    static constexpr int kBytes = 1;
    static constexpr float kTop = 127.0f;
    // The nearest integer of |v| <= 127, ties to even, in the low byte: the sum
    // with 1.5 * 2^23 has it in its last bits (a conversion instruction runs at
    // a quarter of the rate of an addition).
    static __device__ __forceinline__ uint32_t put(float v) {
        return __float_as_uint(__fadd_rn(v, 12582912.0f));
    }
    static __device__ __forceinline__ float get(uint32_t w) {
        return static_cast<float>(static_cast<int8_t>(w & 0xffu));
    }
};

// V codes of a row, packed into words (or one element).
template <int STORE, int V>
__device__ __forceinline__ void store_codes(char* p, const float* v) {
    using S = Store<STORE>;
    if constexpr (V == 1) {
        if constexpr (S::kBytes == 1) *reinterpret_cast<uint8_t*>(p) = static_cast<uint8_t>(S::put(v[0]) & 0xffu);
        else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(S::put(v[0]));
    } else {
        constexpr int W = V * S::kBytes / 4;
        Words<W> w;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (STORE == ROPE_CACHE_FP8) {
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]),
                                                             __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                             __NV_SATFINITE, __NV_E4M3);
                w.w[i] = lo | (hi << 16);
            } else if constexpr (S::kBytes == 1) {
                w.w[i] = __byte_perm(__byte_perm(S::put(v[4 * i]), S::put(v[4 * i + 1]), 0x0040),
                                     __byte_perm(S::put(v[4 * i + 2]), S::put(v[4 * i + 3]), 0x0040), 0x5410);
            } else {
                w.w[i] = S::put(v[2 * i]) | (S::put(v[2 * i + 1]) << 16);
            }
        }
        st_vec<W>(p, w);
    }
}

template <int STORE, int V>
__device__ __forceinline__ void load_codes(const char* p, float* v) {
    using S = Store<STORE>;
    if constexpr (V == 1) {
        const uint32_t w = S::kBytes == 1 ? *reinterpret_cast<const uint8_t*>(p)
                                          : *reinterpret_cast<const uint16_t*>(p);
        v[0] = S::get(w);
    } else {
        constexpr int W = V * S::kBytes / 4;
        const Words<W> w = ldg_vec<W>(p);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            constexpr int per = 4 / S::kBytes;
            v[i] = S::get(w.w[i / per] >> (8 * S::kBytes * (i % per)));
        }
    }
}

// V elements of a dense row as fp32.
template <typename T, int V>
__device__ __forceinline__ void load_row(const char* p, float* v) {
    if constexpr (V == 1) {
        v[0] = Elem<T>::get(ld_elem_scalar<T, true>(p).w[0]);
    } else {
        constexpr int A = 16 / int(sizeof(T));  // elements per 16-byte access
#pragma unroll
        for (int a = 0; a < V / A; ++a) {
            const Words<4> w = ldg_vec<4>(p + 16 * a);
#pragma unroll
            for (int i = 0; i < A; i += 2)
                Pack<T>::get(&w.w[i * int(sizeof(T)) / 4], v[a * A + i], v[a * A + i + 1]);
        }
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_row(char* p, const float* v) {
    if constexpr (V == 1) {
        Words<1> w;
        w.w[0] = Elem<T>::put(v[0]);
        st_elem_scalar<T>(p, w);
    } else {
        constexpr int A = 16 / int(sizeof(T));
#pragma unroll
        for (int a = 0; a < V / A; ++a) {
            Words<4> w;
#pragma unroll
            for (int i = 0; i < A; i += 2)
                Pack<T>::put(&w.w[i * int(sizeof(T)) / 4], v[a * A + i], v[a * A + i + 1]);
            st_vec<4>(p + 16 * a, w);
        }
    }
}

// Where a work row lies.
struct RowAt {
    const CacheSide* side;
    char* dense;
    char* codes;
    float* scale;
    uint32_t tok;
    bool keys;
    bool there;  // the slot is one of the cache's
};

__device__ __forceinline__ RowAt locate(const CacheArgs& a, uint32_t row) {
    RowAt r;
    uint32_t h;
    a.div_rows.divmod(row, r.tok, h);
    const bool second = h >= uint32_t(a.heads);
    if (second) h -= a.heads;
    const int which = second ? 1 : a.first;
    r.side = &a.side[which];
    r.keys = which == 0;
    const uint64_t slot = static_cast<uint64_t>(__ldg(reinterpret_cast<const long long*>(a.slots) + r.tok));
    r.dense = r.side->rows + int64_t(r.tok) * r.side->row_tok + int64_t(h) * r.side->row_head;
    r.there = slot < a.total;  // a negative slot is a huge unsigned one
    uint64_t page = 0, off = 0;
    if (r.there) {
        if (a.total <= 0xffffffffull) {
            page = a.div_page.div(uint32_t(slot));
        } else {
            page = slot / uint64_t(a.page_size);
        }
        off = slot - page * uint64_t(a.page_size);
    }
    r.codes = r.side->codes + int64_t(page) * r.side->page + int64_t(off) * r.side->tok +
              int64_t(h) * r.side->head;
    r.scale = r.side->scale ? r.side->scale + int64_t(page) * r.side->s_page +
                                  int64_t(off) * r.side->s_tok + int64_t(h) * r.side->s_head
                            : nullptr;
    return r;
}

// Turn the V elements of a key row that start at lane j0 (forward rotation).
template <typename T, int V, bool TURN>
__device__ __forceinline__ void turn(const CacheArgs& a, const RowAt& r, int j0, float* v) {
    constexpr int e = int(sizeof(T));
    const char* cos = a.cos + int64_t(r.tok) * a.cos_tok;
    const char* sin = a.sin + int64_t(r.tok) * a.sin_tok;
    const int L = 2 * a.half;
    if constexpr (TURN) {
        // whole accesses lie inside or outside the slice, and so do partners
        const int j = j0 - a.start;
        if (j < 0 || j >= L) return;
        float c[V], s[V];
        load_row<T, V>(cos + j * e, c);
        load_row<T, V>(sin + j * e, s);
        if (a.half_mode) {
            const bool lower = j < a.half;
            float x[V];
            load_row<T, V>(r.dense + (lower ? j0 + a.half : j0 - a.half) * e, x);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float p = __fmul_rn(v[i], c[i]), q = __fmul_rn(x[i], s[i]);
                v[i] = lower ? __fsub_rn(p, q) : __fadd_rn(p, q);
            }
        } else if constexpr (V > 1) {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                float y0, y1;
                rotate_pair<kFwd>(v[i], v[i + 1], c[i], c[i + 1], s[i], s[i + 1], y0, y1);
                v[i] = y0;
                v[i + 1] = y1;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = j0 + i - a.start;
            if (j < 0 || j >= L) continue;
            const bool lower = a.half_mode ? j < a.half : (j & 1) == 0;
            const int partner = a.half_mode ? (lower ? j + a.half : j - a.half) : (j ^ 1);
            float x, c, s;
            load_row<T, 1>(r.dense + (a.start + partner) * e, &x);
            load_row<T, 1>(cos + j * e, &c);
            load_row<T, 1>(sin + j * e, &s);
            const float p = __fmul_rn(v[i], c), q = __fmul_rn(x, s);
            v[i] = lower ? __fsub_rn(p, q) : __fadd_rn(p, q);
        }
    }
}

template <typename T, int STORE, int V, int LANES, int CHUNKS, bool TURN>
__global__ void __launch_bounds__(kCacheThreads)
rope_cache_write_kernel(const __grid_constant__ CacheArgs a) {
    using S = Store<STORE>;
    enter_after_predecessor();
    const uint64_t t = uint64_t(blockIdx.x) * kCacheThreads + threadIdx.x;
    const uint32_t lane = threadIdx.x % LANES;
    const uint64_t row = t / LANES;
    if (row >= a.rows) return;  // whole rows: the lanes of one leave together
    const RowAt r = locate(a, uint32_t(row));

    // the row is loaded and turned whether or not its slot is one of the
    // cache's: its loads need not wait for the slot's
    float v[CHUNKS][V];
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
        const int j = (i * LANES + int(lane)) * V;
        if (j < r.side->dim) load_row<T, V>(r.dense + int64_t(j) * int(sizeof(T)), v[i]);
    }
    if (r.keys && a.half) {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int j = (i * LANES + int(lane)) * V;
            if (j < r.side->dim) turn<T, V, TURN>(a, r, j, v[i]);
        }
    }
    float inv = 1.0f;
    bool finite = true;
    if constexpr (S::kBytes == 1) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i)
            if ((i * LANES + int(lane)) * V < r.side->dim) {
#pragma unroll
                for (int k = 0; k < V; ++k) most = max(most, __float_as_uint(v[i][k]) & 0x7fffffffu);
            }
        const uint32_t mask = LANES == 32 ? 0xffffffffu
                                          : ((1u << LANES) - 1u) << (threadIdx.x % 32 / LANES * LANES);
#pragma unroll
        for (int d = LANES / 2; d; d /= 2) most = max(most, __shfl_xor_sync(mask, most, d));
        finite = most < 0x7f800000u;
        const float m = fmaxf(__uint_as_float(most), 7.8886090522101181e-31f);  // 2^-100
        inv = __fdiv_rn(S::kTop, m);
        if (lane == 0 && r.there) *r.scale = finite ? __fdiv_rn(m, S::kTop) : __uint_as_float(0x7fffffffu);
    }
    if (!r.there) return;
    if (!finite) {  // rare
        inv = 0.0f;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) v[i][k] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
        const int j = (i * LANES + int(lane)) * V;
        if (j >= r.side->dim) continue;
        if constexpr (S::kBytes == 1) {
#pragma unroll
            for (int k = 0; k < V; ++k) v[i][k] = __fmul_rn(v[i][k], inv);
        }
        store_codes<STORE, V>(r.codes + int64_t(j) * S::kBytes, v[i]);
    }
}

template <typename T, int STORE, int V, int LANES, int CHUNKS>
__global__ void __launch_bounds__(kCacheThreads)
rope_cache_read_kernel(const __grid_constant__ CacheArgs a) {
    using S = Store<STORE>;
    enter_after_predecessor();
    const uint64_t t = uint64_t(blockIdx.x) * kCacheThreads + threadIdx.x;
    const uint32_t lane = threadIdx.x % LANES;
    const uint64_t row = t / LANES;
    if (row >= a.rows) return;
    const RowAt r = locate(a, uint32_t(row));
    float v[CHUNKS][V], scale = 1.0f;
    if constexpr (S::kBytes == 1) {
        if (r.there) scale = __ldg(r.scale);
    }
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
        const int j = (i * LANES + int(lane)) * V;
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] = 0.0f;
        if (r.there && j < r.side->dim) load_codes<STORE, V>(r.codes + int64_t(j) * S::kBytes, v[i]);
    }
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
        const int j = (i * LANES + int(lane)) * V;
        if (j >= r.side->dim) continue;
        if constexpr (S::kBytes == 1) {
#pragma unroll
            for (int k = 0; k < V; ++k) v[i][k] = r.there ? __fmul_rn(v[i][k], scale) : 0.0f;
        }
        store_row<T, V>(r.dense + int64_t(j) * int(sizeof(T)), v[i]);
    }
}

// ------------------------------------------------------------------------
// kernel selection (instantiated in one .cu per dense type)
// ------------------------------------------------------------------------

template <typename T, int STORE, bool WRITE, int V, int LANES, int CHUNKS>
const void* pick_cache_turn(const CachePlan& p) {
    if constexpr (!WRITE) return reinterpret_cast<const void*>(&rope_cache_read_kernel<T, STORE, V, LANES, CHUNKS>);
    else if constexpr (V == 1)
        return reinterpret_cast<const void*>(&rope_cache_write_kernel<T, STORE, V, LANES, CHUNKS, false>);
    else
        return p.turn ? reinterpret_cast<const void*>(&rope_cache_write_kernel<T, STORE, V, LANES, CHUNKS, true>)
                      : reinterpret_cast<const void*>(&rope_cache_write_kernel<T, STORE, V, LANES, CHUNKS, false>);
}

// Rows of up to 64 / 128 / 192 / 256 / 1024 elements in 8-element accesses (16
// when 8-bit rows are read), or of up to 128 / 1024 in single elements.
template <typename T, int STORE, bool WRITE>
const void* pick_cache_row(const CachePlan& p) {
    if constexpr (!WRITE && Store<STORE>::kBytes == 1) {
        if (p.vec == 16) {
            switch (p.chunks) {
                case 1: return pick_cache_turn<T, STORE, WRITE, 16, 4, 1>(p);
                case 2: return pick_cache_turn<T, STORE, WRITE, 16, 4, 2>(p);
                case 3: return pick_cache_turn<T, STORE, WRITE, 16, 4, 3>(p);
                default: return pick_cache_turn<T, STORE, WRITE, 16, 4, 4>(p);
            }
        }
    }
    if (p.vec == 8) {
        if (p.lanes == 32) return pick_cache_turn<T, STORE, WRITE, 8, 32, 4>(p);
        switch (p.chunks) {
            case 1: return pick_cache_turn<T, STORE, WRITE, 8, 8, 1>(p);
            case 2: return pick_cache_turn<T, STORE, WRITE, 8, 8, 2>(p);
            case 3: return pick_cache_turn<T, STORE, WRITE, 8, 8, 3>(p);
            default: return pick_cache_turn<T, STORE, WRITE, 8, 8, 4>(p);
        }
    }
    return p.chunks <= 4 ? pick_cache_turn<T, STORE, WRITE, 1, 32, 4>(p)
                         : pick_cache_turn<T, STORE, WRITE, 1, 32, 32>(p);
}

template <typename T, bool WRITE>
const void* pick_cache(const CachePlan& p) {
    switch (p.store) {
        case ROPE_CACHE_BF16: return pick_cache_row<T, ROPE_CACHE_BF16, WRITE>(p);
        case ROPE_CACHE_FP16: return pick_cache_row<T, ROPE_CACHE_FP16, WRITE>(p);
        case ROPE_CACHE_FP8: return pick_cache_row<T, ROPE_CACHE_FP8, WRITE>(p);
        case ROPE_CACHE_INT8: return pick_cache_row<T, ROPE_CACHE_INT8, WRITE>(p);
        default: return nullptr;
    }
}

// defined in rope_cache_{bf16,fp16,fp32}.cu
const void* cache_kernel_bf16(const CachePlan& p, bool write);
const void* cache_kernel_fp16(const CachePlan& p, bool write);
const void* cache_kernel_fp32(const CachePlan& p, bool write);

}  // namespace rope
