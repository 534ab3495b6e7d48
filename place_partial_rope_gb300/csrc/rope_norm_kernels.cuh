// rope_norm_kernels.cuh -- norm and rotation of rows in one pass, and its backward.
//
// Mathematics, per row x (one token, one head) in fp32, n normed lanes:
//   forward   r = 1 / sqrt(eps + sum x_j^2 / n); y_j = (x_j r) w_j, or x_j outside
//             the normed lanes; out = y with its slice rotated, rounded once.
//   backward  g = the transposed rotation of the gradient; u_j = x_j r;
//             t = sum_j w_j g_j u_j; out_j = r (w_j g_j - u_j t / n), or g_j
//             outside; the weight's gradient is the sum of g_j u_j over all rows.
//
// What bounds it: HBM, one pass over the rows; beside it the issue of instructions (2.3 of 4 a
// cycle).  16384 tokens of 32 + 8 heads of 128 bf16: 63 us, 5.4 TB/s (0.79 of what a copy
// reaches); 16411 rows of 576: 13.2 us, 0.47, a call too short for more; backward of 16384 tokens
// of 16 + 4 heads: 59 us, 0.64.  A row is spread over 4 to 32 lanes
// of a warp in chunks of 16 bytes that stay in registers between the sum and the
// store, so it is read once; as many lanes as its chunks take, so that few idle.
// Several heads of a token share a thread's cosines, sines and weights.
// Fast kernels (see there) are for rows whose chunks are normed, and turned, as a whole, and
// whose pairs lie within a chunk (kTurnNear: even starts, adjacent lanes; kTurnPairs: the
// slice's ends and tables pair by pair) or whose partners are a chunk of another lane
// (kTurnFar), which is loaded once more (from L1, before anything of the row is stored, as
// out may be x).  The general ones (kTurnAny) look each element's partner up by itself.  Rows
// that 16-byte accesses do not fit go one element an access.
//
// The backward's blocks stay and walk over the rows: a thread has the same lanes in
// each, keeps their sums of the weight's gradient in registers, and a block writes
// one row of sums, which rope_norm_join_kernel adds up in a fixed order.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <string.h>

#include "rope_f32x2.cuh"
#include "rope_kernels.cuh"
#include "rope_norm.h"

namespace rope {

template <typename T>
struct Chunk {
    static constexpr int VE = 16 / int(sizeof(T));

    static __device__ __forceinline__ void get(const Words<4>& w, float* f) {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            Pack<T>::get(w.w + i * Pack<T>::kWordsPerPair, f[2 * i], f[2 * i + 1]);
    }

    static __device__ __forceinline__ Words<4> put(const float* f) {
        Words<4> w;
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) Pack<T>::put(w.w + i * Pack<T>::kWordsPerPair, f[2 * i], f[2 * i + 1]);
        return w;
    }

    // Puts the bits of one element at place i of a chunk.
    static __device__ __forceinline__ void set(Words<4>& w, int i, uint32_t bits) {
        if constexpr (sizeof(T) == 4) w.w[i] = bits;
        else w.w[i / 2] = i % 2 ? (w.w[i / 2] & 0xffffu) | (bits << 16) : (w.w[i / 2] & 0xffff0000u) | (bits & 0xffffu);
    }

    static __device__ __forceinline__ uint32_t bits(const Words<4>& w, int i) {
        if constexpr (sizeof(T) == 4) return w.w[i];
        else return i % 2 ? w.w[i / 2] >> 16 : w.w[i / 2] & 0xffffu;
    }

    static __device__ __forceinline__ uint32_t element(const char* p) {
        if constexpr (sizeof(T) == 4) return *reinterpret_cast<const volatile uint32_t*>(p);
        else return *reinterpret_cast<const volatile unsigned short*>(p);
    }

    // The elements [e, e + VE) of a row of D; those past its end are zeros.
    static __device__ __forceinline__ Words<4> load(const char* row, int e, int D, bool wide) {
        Words<4> w{};
        if (wide) {
            if (e < D) w = ld_vec<4>(row + e * int(sizeof(T)));
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (e + i < D) set(w, i, element(row + (e + i) * int(sizeof(T))));
        }
        return w;
    }

    static __device__ __forceinline__ void store(char* row, int e, int D, bool wide, const Words<4>& w) {
        if (wide) {
            if (e < D) st_vec<4>(row + e * int(sizeof(T)), w);
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (e + i < D) st_elem_scalar<T>(row + (e + i) * int(sizeof(T)), Words<1>{{bits(w, i)}});
        }
    }
};

// What a lane knows of the chunk from element e on.
template <typename T>
struct NormAt {
    static constexpr int VE = Chunk<T>::VE;
    const NormArgs& a;
    int e;
    bool all, any;  // of its elements are normed

    __device__ __forceinline__ NormAt(const NormArgs& args, int at) : a(args), e(at) {
        all = e >= a.n0 && e + VE <= a.n1;
        any = e + VE > a.n0 && e < a.n1;
    }

    __device__ __forceinline__ bool normed(int i) const { return all || (any && e + i >= a.n0 && e + i < a.n1); }

    __device__ __forceinline__ bool turned(int i) const { return e + i >= a.start && e + i < a.end; }

    // The slice's lane j's partner, and whether j is the first of the two.
    static __device__ __forceinline__ int partner(int j, int half, bool interleave) {
        return interleave ? j ^ 1 : j < half ? j + half : j - half;
    }
};

// Weights of the elements [e, e + VE); 1 outside the normed lanes.
template <typename T>
__device__ __forceinline__ void norm_weights(const NormArgs& a, const char* weight, int e, float* w) {
#pragma unroll
    for (int i = 0; i < Chunk<T>::VE; ++i) {
        w[i] = 1.0f;
        if (!weight || e + i < a.n0 || e + i >= a.n1) continue;
        const int at = e + i - a.n0;
        if (a.weight32) w[i] = __ldg(reinterpret_cast<const float*>(weight) + at);
        else w[i] = Elem<T>::get(ld_elem_scalar<T, true>(weight + int64_t(at) * int(sizeof(T))).w[0]);
    }
}

// A table's row at the slice's lanes [e - start, ...) of a chunk; 0 outside the slice.
template <typename T>
__device__ __forceinline__ void norm_table(const NormArgs& a, const char* row, int e, float* f) {
#pragma unroll
    for (int i = 0; i < Chunk<T>::VE; ++i) {
        f[i] = 0.0f;
        if (e + i >= a.start && e + i < a.end)
            f[i] = Elem<T>::get(ld_elem_scalar<T, true>(row + (e + i - a.start) * int(sizeof(T))).w[0]);
    }
}

// The partners of a chunk's elements, gathered one by one: a row's values, the weights, or a
// table's values; 0 (weights: 1) outside the slice.
template <typename T>
struct NormFar {
    static constexpr int VE = Chunk<T>::VE;

    static __device__ __forceinline__ Words<4> load(const NormArgs& a, const char* row, int e) {
        Words<4> w{};
        const int half = (a.end - a.start) / 2;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const int j = e + i - a.start;
            if (j >= 0 && j < 2 * half)
                Chunk<T>::set(w, i, Chunk<T>::element(row + (a.start + NormAt<T>::partner(j, half, a.interleave)) *
                                                                int(sizeof(T))));
        }
        return w;
    }

    static __device__ __forceinline__ void weights(const NormArgs& a, const char* weight, int e, float* w) {
        const int half = (a.end - a.start) / 2;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            w[i] = 1.0f;
            const int j = e + i - a.start;
            if (!weight || j < 0 || j >= 2 * half) continue;
            const int k = a.start + NormAt<T>::partner(j, half, a.interleave) - a.n0;
            if (k < 0 || k >= a.n1 - a.n0) continue;
            if (a.weight32) w[i] = __ldg(reinterpret_cast<const float*>(weight) + k);
            else w[i] = Elem<T>::get(ld_elem_scalar<T, true>(weight + int64_t(k) * int(sizeof(T))).w[0]);
        }
    }

    static __device__ __forceinline__ void table(const NormArgs& a, const char* row, int e, float* f) {
        const int half = (a.end - a.start) / 2;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            f[i] = 0.0f;
            const int j = e + i - a.start;
            if (j >= 0 && j < 2 * half)
                f[i] = Elem<T>::get(
                    ld_elem_scalar<T, true>(row + NormAt<T>::partner(j, half, a.interleave) * int(sizeof(T))).w[0]);
        }
    }
};

// An item's rows: U heads from h of a token.
struct NormItem {
    uint32_t b, s, tok;
    int h;

    __device__ __forceinline__ NormItem(const NormArgs& a, const NormRows& r, uint32_t item, int U) {
        uint32_t hg;
        r.div_groups.divmod(item, tok, hg);
        a.div_S.divmod(tok, b, s);
        h = int(hg) * U;
    }

    __device__ __forceinline__ int64_t at(const int64_t* st) const { return b * st[0] + s * st[1] + h * st[2]; }
};

template <typename T, int C, int U>
__device__ __forceinline__ void norm_fwd_item(const NormArgs& a, const NormRows& r, uint32_t item, bool live, int p,
                                              int P) {
    constexpr int VE = Chunk<T>::VE;
    using Far = NormFar<T>;
    const NormItem at(a, r, live ? item : 0, U);
    const char* x = r.x + at.at(r.x_st);
    char* out = r.out + at.at(r.out_st);
    Words<4> own[U][C], other[U][C];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool on = live && at.h + u < r.heads;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * P + p) * VE;
            own[u][c] = Words<4>{};
            if (on) own[u][c] = Chunk<T>::load(x + u * r.x_st[2], e, a.D, a.wide);
            other[u][c] = Words<4>{};
            if (on) other[u][c] = Far::load(a, x + u * r.x_st[2], e);
        }
    }
    float sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        sum[u] = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const NormAt<T> n(a, (c * P + p) * VE);
            float f[VE];
            Chunk<T>::get(own[u][c], f);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (n.normed(i)) sum[u] = fmaf(f[i], f[i], sum[u]);
        }
    }
    for (int d = P / 2; d; d /= 2)
#pragma unroll
        for (int u = 0; u < U; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], d);
    __syncwarp();  // the warp's loads come before its stores: out may be x
    if (!live) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        sum[u] = __frsqrt_rn(fmaf(sum[u], a.inv_n, a.eps));
        if (r.rstd && p == 0 && at.h + u < r.heads) r.rstd[int64_t(at.tok) * r.heads + at.h + u] = sum[u];
    }
    const char* cos = a.cos + at.b * a.cos_st[0] + at.s * a.cos_st[1];
    const char* sin = a.sin + at.b * a.sin_st[0] + at.s * a.sin_st[1];
    const int half = (a.end - a.start) / 2;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const NormAt<T> n(a, (c * P + p) * VE);
        if (n.e >= a.D) continue;
        const bool turns = n.e + VE > a.start && n.e < a.end;
        float w[VE], wo[VE], cs[VE], sn[VE];
        norm_weights<T>(a, r.weight, n.e, w);
        if (turns) {
            norm_table<T>(a, cos, n.e, cs);
            norm_table<T>(a, sin, n.e, sn);
            Far::weights(a, r.weight, n.e, wo);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (at.h + u >= r.heads) continue;
            float f[VE];
            Chunk<T>::get(own[u][c], f);
#pragma unroll
            for (int i = 0; i < VE; ++i) f[i] = f[i] * (n.normed(i) ? sum[u] : 1.0f) * w[i];
            if (turns) {
                float g[VE];
                Chunk<T>::get(other[u][c], g);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    if (!n.turned(i)) continue;
                    const int j = n.e + i - a.start, k = a.start + NormAt<T>::partner(j, half, a.interleave);
                    const float y = g[i] * (k >= a.n0 && k < a.n1 ? sum[u] : 1.0f) * wo[i];
                    const bool first = a.interleave ? j % 2 == 0 : j < half;
                    f[i] = __fadd_rn(__fmul_rn(f[i], cs[i]), __fmul_rn(first ? -y : y, sn[i]));
                }
            }
            Chunk<T>::store(out + u * r.out_st[2], n.e, a.D, a.wide, Chunk<T>::put(f));
        }
    }
}

template <typename T, int C, int U>
__global__ void __launch_bounds__(kNormThreads) rope_norm_fwd_kernel(const __grid_constant__ NormArgs a) {
    enter_after_predecessor();
    const int P = 1 << a.lanes_log2, p = int(threadIdx.x) & (P - 1);
    uint32_t item = blockIdx.x * uint32_t(kNormThreads >> a.lanes_log2) + (threadIdx.x >> a.lanes_log2);
    const bool second = a.sides == 2 && item >= a.side[0].items;
    if (second) item -= a.side[0].items;
    const NormRows& r = a.side[second ? 1 : 0];
    norm_fwd_item<T, C, U>(a, r, item, item < r.items, p, P);
}

// One item of the backward; the thread's sums of the weight's gradient go on in dw.
template <typename T, int C, int U>
__device__ __forceinline__ void norm_bwd_item(const NormArgs& a, const NormRows& r, uint32_t item, bool live, int p,
                                              int P, const float (*w)[Chunk<T>::VE], float (*dw)[Chunk<T>::VE]) {
    constexpr int VE = Chunk<T>::VE;
    using Far = NormFar<T>;
    const NormItem at(a, r, live ? item : 0, U);
    const char* x = r.x + at.at(r.x_st);
    const char* grad = r.grad + at.at(r.grad_st);
    char* out = r.out + at.at(r.out_st);
    Words<4> own[U][C], in[U][C], other[U][C];
    float rstd[U], t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool on = live && at.h + u < r.heads;
        rstd[u] = on ? __ldg(r.rstd + int64_t(at.tok) * r.heads + at.h + u) : 0.0f;
        t[u] = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * P + p) * VE;
            own[u][c] = in[u][c] = Words<4>{};
            if (on) {
                in[u][c] = Chunk<T>::load(x + u * r.x_st[2], e, a.D, a.wide);
                own[u][c] = Chunk<T>::load(grad + u * r.grad_st[2], e, a.D, a.wide);
            }
            other[u][c] = Words<4>{};
            if (on) other[u][c] = Far::load(a, grad + u * r.grad_st[2], e);
        }
    }
    const char* cos = a.cos + at.b * a.cos_st[0] + at.s * a.cos_st[1];
    const char* sin = a.sin + at.b * a.sin_st[0] + at.s * a.sin_st[1];
    const int half = (a.end - a.start) / 2;
    float g[U][C][VE];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const NormAt<T> n(a, (c * P + p) * VE);
        const bool turns = n.e + VE > a.start && n.e < a.end;
        float cs[VE], sn[VE];
        if (turns) {
            norm_table<T>(a, cos, n.e, cs);
            Far::table(a, sin, n.e, sn);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float* f = g[u][c];
            Chunk<T>::get(own[u][c], f);
            if (turns) {
                float o[VE];
                Chunk<T>::get(other[u][c], o);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    if (!n.turned(i)) continue;
                    const int j = n.e + i - a.start;
                    const bool first = a.interleave ? j % 2 == 0 : j < half;
                    f[i] = __fadd_rn(__fmul_rn(f[i], cs[i]), __fmul_rn(first ? o[i] : -o[i], sn[i]));
                }
            }
            float v[VE];
            Chunk<T>::get(in[u][c], v);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                if (!n.normed(i)) continue;
                const float gu = f[i] * (v[i] * rstd[u]);
                dw[c][i] += gu;  // 0 for a row that is not there
                t[u] = fmaf(w[c][i], gu, t[u]);
            }
        }
    }
    for (int d = P / 2; d; d /= 2)
#pragma unroll
        for (int u = 0; u < U; ++u) t[u] += __shfl_xor_sync(0xffffffffu, t[u], d);
    __syncwarp();  // the warp's loads come before its stores: out may be grad
    if (!live) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (at.h + u >= r.heads) continue;
        const float mean = t[u] * a.inv_n;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const NormAt<T> n(a, (c * P + p) * VE);
            if (n.e >= a.D) continue;
            float v[VE], y[VE];
            Chunk<T>::get(in[u][c], v);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                y[i] = n.normed(i) ? rstd[u] * fmaf(w[c][i], g[u][c][i], -(v[i] * rstd[u]) * mean) : g[u][c][i];
            Chunk<T>::store(out + u * r.out_st[2], n.e, a.D, a.wide, Chunk<T>::put(y));
        }
    }
}

template <typename T, int C, int U>
__global__ void __launch_bounds__(kNormThreads) rope_norm_bwd_kernel(const __grid_constant__ NormArgs a) {
    constexpr int VE = Chunk<T>::VE, WARPS = kNormThreads / 32;
    __shared__ float sums[WARPS][32 * C * VE];
    enter_after_predecessor();
    const int P = 1 << a.lanes_log2, p = int(threadIdx.x) & (P - 1), lane = int(threadIdx.x) & 31;
    const uint32_t per = uint32_t(kNormThreads >> a.lanes_log2);
    for (int side = 0; side < a.sides; ++side) {
        const NormRows& r = a.side[side];
        float w[C][VE], dw[C][VE];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            norm_weights<T>(a, r.weight, (c * P + p) * VE, w[c]);
#pragma unroll
            for (int i = 0; i < VE; ++i) dw[c][i] = 0.0f;
        }
        // (blocks x their items stay below 2^32: items < 2^31)
        for (uint32_t first = blockIdx.x * per; first < r.items; first += gridDim.x * per) {
            const uint32_t item = first + (threadIdx.x >> a.lanes_log2);
            norm_bwd_item<T, C, U>(a, r, item, item < r.items, p, P, w, dw);
        }
        if (!r.part) continue;
        for (int d = P; d < 32; d *= 2)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < VE; ++i) dw[c][i] += __shfl_xor_sync(0xffffffffu, dw[c][i], d);
        if (lane < P)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < VE; ++i) sums[threadIdx.x >> 5][(c * P + p) * VE + i] = dw[c][i];
        __syncthreads();
        for (int e = a.n0 + int(threadIdx.x); e < a.n1; e += kNormThreads) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) s += sums[k][e];
            r.part[int64_t(blockIdx.x) * (a.n1 - a.n0) + e - a.n0] = s;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------
// rows whose chunks are each normed or not, and turned or not (kTurnPairs: pair by pair)
// ------------------------------------------------------------------------

// The general kernels ask for each element whether it is normed and turned, and were bound by
// that: 270 instructions a chunk.  Here a chunk's arithmetic is on pairs of fp32 numbers,
// and weights go into the tables once for all heads of a token.
template <typename T>
struct NormPairs {
    static constexpr int VE = Chunk<T>::VE, N = VE / 2;

    static __device__ __forceinline__ void get(const Words<4>& w, float2* f) {
#pragma unroll
        for (int i = 0; i < N; ++i) Pack<T>::get(w.w + i * Pack<T>::kWordsPerPair, f[i].x, f[i].y);
    }
    static __device__ __forceinline__ Words<4> put(const float2* f) {
        Words<4> w;
#pragma unroll
        for (int i = 0; i < N; ++i) Pack<T>::put(w.w + i * Pack<T>::kWordsPerPair, f[i].x, f[i].y);
        return w;
    }

    // Weights of a chunk that is normed as a whole; else 1.
    static __device__ __forceinline__ void weights(const NormArgs& a, const char* weight, int e, bool normed, float2* w) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = make_float2(1.0f, 1.0f);
        if (!normed || !weight) return;
        if (a.weight32) {
            const float4* p = reinterpret_cast<const float4*>(weight + int64_t(e - a.n0) * 4);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float4 q = __ldg(p + i / 2);
                w[i] = make_float2(q.x, q.y);
                w[i + 1] = make_float2(q.z, q.w);
            }
        } else {
            get(ldg_vec<4>(weight + int64_t(e - a.n0) * int(sizeof(T))), w);
        }
    }

    // A table's pairs from element e of the row on; kTurnPairs: those inside the slice.
    template <int TURN>
    static __device__ __forceinline__ void table(const NormArgs& a, const char* row, int e, float2* f) {
        if constexpr (TURN != kTurnPairs) {
            get(ldg_vec<4>(row + (e - a.start) * int(sizeof(T))), f);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int j = e + 2 * i - a.start;
                f[i] = make_float2(0.0f, 0.0f);
                if (j < 0 || j >= a.end - a.start) continue;
                const char* p = row + j * int(sizeof(T));
                constexpr int W = Pack<T>::kWordsPerPair;
                const Words<W> w = a.pairs_cs ? ldg_vec<W>(p) : ld_pair_scalar<T, true>(p);
                Pack<T>::get(w.w, f[i].x, f[i].y);
            }
        }
    }
};

__device__ __forceinline__ float2 swapped(float2 x) { return make_float2(x.y, x.x); }

template <typename T, int C, int U, int TURN>
__global__ void __launch_bounds__(kNormThreads) rope_norm_fast_fwd_kernel(const __grid_constant__ NormArgs a) {
    using N = NormPairs<T>;
    constexpr int VE = N::VE, H = N::N;
    constexpr bool FAR = TURN == kTurnFar, PARTS = TURN == kTurnPairs;
    enter_after_predecessor();
    const int P = 1 << a.lanes_log2, p = int(threadIdx.x) & (P - 1);
    uint32_t item = blockIdx.x * uint32_t(kNormThreads >> a.lanes_log2) + (threadIdx.x >> a.lanes_log2);
    const bool second = a.sides == 2 && item >= a.side[0].items;
    if (second) item -= a.side[0].items;
    const NormRows& r = a.side[second ? 1 : 0];
    const bool live = item < r.items;
    const NormItem at(a, r, live ? item : 0, U);
    const char* x = r.x + at.at(r.x_st);
    char* out = r.out + at.at(r.out_st);
    const int half = (a.end - a.start) / 2;
    Words<4> own[U][C], other[FAR ? U : 1][FAR ? C : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool on = live && at.h + u < r.heads;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * P + p) * VE;
            own[u][c] = Words<4>{};
            if (on && e < a.D) own[u][c] = ld_vec<4>(x + u * r.x_st[2] + e * int(sizeof(T)));
            if constexpr (FAR) {
                other[u][c] = Words<4>{};
                if (on && e >= a.start && e < a.end)
                    other[u][c] = ld_vec<4>(x + u * r.x_st[2] + (e < a.start + half ? e + half : e - half) * int(sizeof(T)));
            }
        }
    }
    float sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * P + p) * VE;
            float2 f[H];
            N::get(own[u][c], f);
            if (e >= a.n0 && e < a.n1)
#pragma unroll
                for (int i = 0; i < H; ++i) t = fma2(f[i], f[i], t);
        }
        sum[u] = t.x + t.y;
    }
    for (int d = P / 2; d; d /= 2)
#pragma unroll
        for (int u = 0; u < U; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], d);
    __syncwarp();  // the warp's loads come before its stores: out may be x
    if (!live) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        sum[u] = __frsqrt_rn(fmaf(sum[u], a.inv_n, a.eps));
        if (r.rstd && p == 0 && at.h + u < r.heads) r.rstd[int64_t(at.tok) * r.heads + at.h + u] = sum[u];
    }
    const char* cos = a.cos + at.b * a.cos_st[0] + at.s * a.cos_st[1];
    const char* sin = a.sin + at.b * a.sin_st[0] + at.s * a.sin_st[1];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (c * P + p) * VE;
        if (e >= a.D) continue;
        const bool normed = e >= a.n0 && e < a.n1, turned = e + (PARTS ? VE - 1 : 0) >= a.start && e < a.end;
        float2 w[H], ws[H];
        N::weights(a, r.weight, e, normed, w);
        uint32_t in = 0;  // pairs that turn
        if (turned) {
            // w cos for an element, and for its partner w sin with the rotation's sign
            float2 cs[H], sn[H], wo[H];
            N::template table<TURN>(a, cos, e, cs);
            N::template table<TURN>(a, sin, e, sn);
            if constexpr (FAR) N::weights(a, r.weight, e < a.start + half ? e + half : e - half, normed, wo);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const bool on = !PARTS || (e + 2 * i >= a.start && e + 2 * i < a.end);
                if (on) in |= 1u << i;
                if constexpr (FAR) {
                    const float sign = e < a.start + half ? -1.0f : 1.0f;
                    ws[i] = mul2(mul2(wo[i], sn[i]), make_float2(sign, sign));
                } else {
                    ws[i] = mul2(swapped(w[i]), make_float2(-sn[i].x, sn[i].y));
                }
                if (on) w[i] = mul2(w[i], cs[i]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (at.h + u >= r.heads) continue;
            const float by = normed ? sum[u] : 1.0f;
            float2 f[H], g[H];
            N::get(own[u][c], f);
            if (turned) {
                if constexpr (FAR) N::get(other[u][c], g);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float2 y = mul2(f[i], w[i]);
                    const float2 z = fma2(FAR ? g[i] : swapped(f[i]), ws[i], y);
                    f[i] = !PARTS || (in >> i & 1u) ? z : y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < H; ++i) f[i] = mul2(f[i], w[i]);
            }
#pragma unroll
            for (int i = 0; i < H; ++i) f[i] = mul2(f[i], make_float2(by, by));
            st_vec<4>(out + u * r.out_st[2] + e * int(sizeof(T)), N::put(f));
        }
    }
}

// (16-bit rows of one chunk a lane: three blocks an SM, at 80 registers, 59 us for 16384 tokens
// of 16 + 4 heads of 128, where 118 registers and two took 70 and 64 and four 71.  0 is no bound:
// 4845 tokens of 12 + 12 heads of 128 fp32 lanes take 36.5 us at 62 registers so, 41 with a
// bound of three and 45 with one of one)
template <typename T, int C, int U, int TURN>
__global__ void __launch_bounds__(kNormThreads, C == 1 && sizeof(T) == 2 ? 3 : 0)
    rope_norm_fast_bwd_kernel(const __grid_constant__ NormArgs a) {
    using N = NormPairs<T>;
    constexpr int VE = N::VE, H = N::N, WARPS = kNormThreads / 32;
    constexpr bool FAR = TURN == kTurnFar, PARTS = TURN == kTurnPairs;
    __shared__ float sums[WARPS][32 * C * VE];
    enter_after_predecessor();
    const int P = 1 << a.lanes_log2, p = int(threadIdx.x) & (P - 1), lane = int(threadIdx.x) & 31;
    const uint32_t per = uint32_t(kNormThreads >> a.lanes_log2);
    const int half = (a.end - a.start) / 2;
    for (int side = 0; side < a.sides; ++side) {
        const NormRows& r = a.side[side];
        float2 w[C][H], dw[C][H];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * P + p) * VE;
            N::weights(a, r.weight, e, e >= a.n0 && e < a.n1, w[c]);
#pragma unroll
            for (int i = 0; i < H; ++i) dw[c][i] = make_float2(0.0f, 0.0f);
        }
        for (uint32_t first = blockIdx.x * per; first < r.items; first += gridDim.x * per) {
            const uint32_t item = first + (threadIdx.x >> a.lanes_log2);
            const bool live = item < r.items;
            const NormItem at(a, r, live ? item : 0, U);
            const char* x = r.x + at.at(r.x_st);
            const char* grad = r.grad + at.at(r.grad_st);
            char* out = r.out + at.at(r.out_st);
            Words<4> own[U][C], in[U][C], other[FAR ? U : 1][FAR ? C : 1];
            float rstd[U], t[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool on = live && at.h + u < r.heads;
                rstd[u] = on ? __ldg(r.rstd + int64_t(at.tok) * r.heads + at.h + u) : 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int e = (c * P + p) * VE;
                    own[u][c] = in[u][c] = Words<4>{};
                    if (on && e < a.D) {
                        own[u][c] = ld_vec<4>(grad + u * r.grad_st[2] + e * int(sizeof(T)));
                        in[u][c] = ld_vec<4>(x + u * r.x_st[2] + e * int(sizeof(T)));
                    }
                    if constexpr (FAR) {
                        other[u][c] = Words<4>{};
                        if (on && e >= a.start && e < a.end)
                            other[u][c] = ld_vec<4>(grad + u * r.grad_st[2] +
                                                    (e < a.start + half ? e + half : e - half) * int(sizeof(T)));
                    }
                }
            }
            const char* cos = a.cos + at.b * a.cos_st[0] + at.s * a.cos_st[1];
            const char* sin = a.sin + at.b * a.sin_st[0] + at.s * a.sin_st[1];
            float2 g[U][C][H], t2[U];
#pragma unroll
            for (int u = 0; u < U; ++u) t2[u] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e = (c * P + p) * VE;
                const bool normed = e >= a.n0 && e < a.n1, turned = e + (PARTS ? VE - 1 : 0) >= a.start && e < a.end;
                float2 cs[H], sn[H];
                if (turned) {
                    N::template table<TURN>(a, cos, e, cs);
                    N::template table<TURN>(a, sin, FAR ? (e < a.start + half ? e + half : e - half) : e, sn);
                    const float sign = e < a.start + half ? 1.0f : -1.0f;
#pragma unroll
                    for (int i = 0; i < H; ++i)
                        sn[i] = FAR ? mul2(sn[i], make_float2(sign, sign)) : make_float2(sn[i].y, -sn[i].x);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float2* f = g[u][c];
                    N::get(own[u][c], f);
                    if (turned) {
                        float2 o[H];
                        if constexpr (FAR) N::get(other[u][c], o);
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            const float2 z = fma2(FAR ? o[i] : swapped(f[i]), sn[i], mul2(f[i], cs[i]));
                            if (!PARTS || (e + 2 * i >= a.start && e + 2 * i < a.end)) f[i] = z;
                        }
                    }
                    if (normed) {
                        float2 v[H];
                        N::get(in[u][c], v);
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            const float2 unit = mul2(v[i], make_float2(rstd[u], rstd[u]));
                            dw[c][i] = fma2(f[i], unit, dw[c][i]);  // 0 for a row that is not there
                            f[i] = mul2(f[i], w[c][i]);
                            t2[u] = fma2(f[i], unit, t2[u]);
                        }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) t[u] = t2[u].x + t2[u].y;
            for (int d = P / 2; d; d /= 2)
#pragma unroll
                for (int u = 0; u < U; ++u) t[u] += __shfl_xor_sync(0xffffffffu, t[u], d);
            __syncwarp();  // the warp's loads come before its stores: out may be grad
            if (!live) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (at.h + u >= r.heads) continue;
                // r (w g - u t / n), with u = x r
                const float by = -(t[u] * a.inv_n) * rstd[u];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int e = (c * P + p) * VE;
                    if (e >= a.D) continue;
                    float2* f = g[u][c];
                    if (e >= a.n0 && e < a.n1) {
                        float2 v[H];
                        N::get(in[u][c], v);
#pragma unroll
                        for (int i = 0; i < H; ++i)
                            f[i] = mul2(fma2(v[i], make_float2(by, by), f[i]), make_float2(rstd[u], rstd[u]));
                    }
                    st_vec<4>(out + u * r.out_st[2] + e * int(sizeof(T)), N::put(f));
                }
            }
        }
        if (!r.part) continue;
        for (int d = P; d < 32; d *= 2)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    dw[c][i].x += __shfl_xor_sync(0xffffffffu, dw[c][i].x, d);
                    dw[c][i].y += __shfl_xor_sync(0xffffffffu, dw[c][i].y, d);
                }
        if (lane < P)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < H; ++i)
                    *reinterpret_cast<float2*>(&sums[threadIdx.x >> 5][(c * P + p) * VE + 2 * i]) = dw[c][i];
        __syncthreads();
        for (int e = a.n0 + int(threadIdx.x); e < a.n1; e += kNormThreads) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) s += sums[k][e];
            r.part[int64_t(blockIdx.x) * (a.n1 - a.n0) + e - a.n0] = s;
        }
        __syncthreads();
    }
}

template <typename T, int C, int U, bool BACK>
NormKernel norm_turn(const NormPlan& p) {
    const void* f;
    if constexpr (BACK) {
        f = p.turn == kTurnNear    ? reinterpret_cast<const void*>(&rope_norm_fast_bwd_kernel<T, C, U, kTurnNear>)
            : p.turn == kTurnPairs ? reinterpret_cast<const void*>(&rope_norm_fast_bwd_kernel<T, C, U, kTurnPairs>)
            : p.turn == kTurnFar   ? reinterpret_cast<const void*>(&rope_norm_fast_bwd_kernel<T, C, U, kTurnFar>)
                                   : reinterpret_cast<const void*>(&rope_norm_bwd_kernel<T, C, U>);
    } else {
        f = p.turn == kTurnNear    ? reinterpret_cast<const void*>(&rope_norm_fast_fwd_kernel<T, C, U, kTurnNear>)
            : p.turn == kTurnPairs ? reinterpret_cast<const void*>(&rope_norm_fast_fwd_kernel<T, C, U, kTurnPairs>)
            : p.turn == kTurnFar   ? reinterpret_cast<const void*>(&rope_norm_fast_fwd_kernel<T, C, U, kTurnFar>)
                                   : reinterpret_cast<const void*>(&rope_norm_fwd_kernel<T, C, U>);
    }
    return NormKernel{f, U};
}

// Heads that a thread takes of a token, where there are that many.
template <typename T, int C, bool BACK>
NormKernel norm_pick(const NormPlan& p) {
    // (two prompts of 8192 tokens, 32 + 8 heads of 128 bf16, 8, 4 and 2 heads: 73, 63.5 and 78 us;
    // backward of 16 + 4 heads, 4, 2 and 1: 84, 70 and 73)
    constexpr int MANY = BACK ? (C == 1 ? 2 : 1) : C == 1 ? 4 : C <= 3 ? 2 : 1;
    return p.many ? norm_turn<T, C, MANY, BACK>(p) : norm_turn<T, C, 1, BACK>(p);
}

}  // namespace rope
