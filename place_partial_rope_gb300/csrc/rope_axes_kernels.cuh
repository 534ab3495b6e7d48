// rope_axes_kernels.cuh -- the positions call with several axes.
//
// Mathematics: pair k of the slice belongs to axis a(k) and turns by
//   theta_k = p[a(k)][b][s] * omega_k,
//   forward  y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin,
//   backward the transpose (sin negated).
// The host makes a(k) and omega_k (two fp32 parts) for the call's sections,
// order and spectrum, so the kernel knows neither: a pair looks both up.
//
// What bounds it: one read and one write of the slice, so HBM; the table is
// 4.6 KB of shared memory a block and the positions 4 bytes per axis and
// token.  The layout of the work is that of rope_partial_pos_kernel (a thread
// owns one access of x in U heads of a token and computes its angles once
// for them).  A thread loads the token's positions on every axis up front
// (at most four loads that a warp shares, in flight with those of x) and picks
// one per pair by two selects, rather than one dependent load per pair.
// Measured: 2 videos of 16 x 30 x 52 patches, 24 heads of 128 bf16 lanes (614 MB),
// 93.2 us, 6.6 TB/s or 0.99 of the measured copy rate; a call on 256 patches
// takes 8 us, the host's time.
#pragma once
#include "rope_axes.h"
#include "rope_kernels.cuh"

namespace rope {

template <typename T, int VEC, bool SCALAR, int U, int DIR, bool HALF>
__global__ void __launch_bounds__(kThreads)
rope_partial_axes_kernel(const KernelArgs a, const __grid_constant__ AxisTable f) {
    __shared__ float w_hi[kMaxPairs];
    __shared__ float w_lo[kMaxPairs];
    __shared__ uint8_t w_axis[kMaxPairs];
    for (int i = threadIdx.x; i < a.pairs; i += kThreads) {
        w_hi[i] = f.hi[i];
        w_lo[i] = f.lo[i];
        w_axis[i] = f.axis[i];
    }
    __syncthreads();

    constexpr int W = VEC >= 4 ? VEC / 4 : 1;
    constexpr int E = VEC / int(sizeof(T)) > 0 ? VEC / int(sizeof(T)) : 1;  // elements per chunk
    constexpr int NA = HALF ? E : (E / 2 > 0 ? E / 2 : 1);                  // angles per chunk

    enter_after_predecessor();
    const uint64_t t = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (t >= a.tasks) return;
    uint32_t rest, c, tok, hg, b, s;
    a.divC.divmod(uint32_t(t), rest, c);
    a.divH.divmod(rest, tok, hg);
    a.divS.divmod(tok, b, s);
    const int n0 = int(hg) * U;
    char* x0 = a.x + int64_t(tok) * a.tok_bytes + int64_t(n0) * a.row_bytes + int64_t(c) * VEC;

    Words<W> xa[U], xb[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (i == 0 || n0 + i < a.N) {
            if constexpr (HALF) {
                xa[i] = load_x_half<T, W, SCALAR>(x0 + i * a.row_bytes);
                xb[i] = load_x_half<T, W, SCALAR>(x0 + i * a.row_bytes + a.half_off);
            } else {
                xa[i] = load_x<T, W, SCALAR>(x0 + i * a.row_bytes);
            }
        }
    }

    const int32_t* pp = a.pos + int64_t(b) * a.pos_b + int64_t(s) * a.pos_s;
    int32_t pos[ROPE_MAX_AXES];
#pragma unroll
    for (int i = 0; i < ROPE_MAX_AXES; ++i) pos[i] = i < f.axes ? __ldg(pp + i * f.pos_a) : 0;

    const int k0 = int(c) * NA;
    float cs[NA], sn[NA];
#pragma unroll
    for (int j = 0; j < NA; ++j) {
        const int ax = w_axis[k0 + j];
        const int32_t lo = ax & 1 ? pos[1] : pos[0], hi = ax & 1 ? pos[3] : pos[2];
        angle_cos_sin(__int2float_rn(ax & 2 ? hi : lo), w_hi[k0 + j], w_lo[k0 + j], cs[j], sn[j]);
    }

#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (i == 0 || n0 + i < a.N) {
            char* xp = x0 + i * a.row_bytes;
            if constexpr (HALF) {
                Words<W> ya, yb;
                rotate_half_angles<T, W, SCALAR, DIR>(xa[i], xb[i], cs, sn, ya, yb);
                store_x_half<T, W, SCALAR>(xp, ya);
                store_x_half<T, W, SCALAR>(xp + a.half_off, yb);
            } else {
                store_x<T, W, SCALAR>(xp, rotate_chunk_angles<T, W, DIR>(xa[i], cs, sn));
            }
        }
    }
}

template <typename T, int VEC, bool SCALAR, int U, bool HALF>
const void* pick_axes_dir(const Plan& p) {
    return p.dir == kFwd
               ? reinterpret_cast<const void*>(&rope_partial_axes_kernel<T, VEC, SCALAR, U, kFwd, HALF>)
               : reinterpret_cast<const void*>(&rope_partial_axes_kernel<T, VEC, SCALAR, U, kBwd, HALF>);
}

template <typename T, int VEC, bool SCALAR, bool HALF>
const void* pick_axes_heads(const Plan& p) {
    switch (p.U) {
        case 1: return pick_axes_dir<T, VEC, SCALAR, 1, HALF>(p);
        case 2: return pick_axes_dir<T, VEC, SCALAR, 2, HALF>(p);
        case 4: return pick_axes_dir<T, VEC, SCALAR, 4, HALF>(p);
        case 8:
            if constexpr (VEC < 16) return pick_axes_dir<T, VEC, SCALAR, 8, HALF>(p);
            else return nullptr;
        default: return nullptr;
    }
}

// The accesses that make_plan() gives a positions call: 16, 8 or 4 bytes, or
// single elements (a pair of them in interleave mode).
template <typename T>
const void* pick_axes(const Plan& p) {
    constexpr int e = int(sizeof(T));
    if (p.half) {
        if (p.path == kScalarPair) {
            if constexpr (e == 2) return pick_axes_heads<T, 2, true, true>(p);
            else return nullptr;  // an fp32 element is a 4-byte chunk
        }
        switch (p.vec) {
            case 16: return pick_axes_heads<T, 16, false, true>(p);
            case 8: return pick_axes_heads<T, 8, false, true>(p);
            case 4: return pick_axes_heads<T, 4, false, true>(p);
            default: return nullptr;
        }
    }
    if (p.path == kScalarPair) return pick_axes_heads<T, 2 * e, true, false>(p);
    switch (p.vec) {
        case 16: return pick_axes_heads<T, 16, false, false>(p);
        case 8: return pick_axes_heads<T, 8, false, false>(p);
        case 4:
            if constexpr (e == 2) return pick_axes_heads<T, 4, false, false>(p);
            else return nullptr;
        default: return nullptr;
    }
}

}  // namespace rope
