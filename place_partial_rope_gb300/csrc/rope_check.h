// rope_check.h -- checks of arguments that the library's host files share: sizes,
// strides, alignment, the cache descriptor, and whether tensors share bytes.
#pragma once
#include <stdint.h>

#include "rope_error.h"
#include "rope_serving.h"

namespace rope {

constexpr int64_t kMaxSize = int64_t(1) << 40;  // of any one size or stride: products of two fit

inline int size_of(int dtype) { return dtype == ROPE_FP32 ? 4 : 2; }

inline bool valid_dtype(int d) { return d == ROPE_BF16 || d == ROPE_FP16 || d == ROPE_FP32; }

inline bool valid_store(int s) {
    return s == ROPE_CACHE_BF16 || s == ROPE_CACHE_FP16 || s == ROPE_CACHE_FP8 ||
           s == ROPE_CACHE_INT8;
}

inline int code_size(int store) { return store == ROPE_CACHE_BF16 || store == ROPE_CACHE_FP16 ? 2 : 1; }

inline bool aligned(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % uint64_t(n) == 0; }

// Elements from the first to the last of a tensor whose last dim (`row`
// elements) is contiguous; -1 when a stride is negative, or smaller than
// `apart` on a dim of more than one, or when the sum is out of range.
inline int64_t span(const int64_t* shape, const int64_t* stride, int n, int64_t row, int64_t apart) {
    int64_t sum = row;
    for (int k = 0; k < n; ++k) {
        if (shape[k] <= 1) continue;
        if (stride[k] < apart || stride[k] < 0 || stride[k] > kMaxSize || shape[k] > kMaxSize)
            return -1;
        if (stride[k] != 0 && shape[k] > (int64_t(1) << 60) / stride[k]) return -1;
        sum += (shape[k] - 1) * stride[k];
        if (sum > (int64_t(1) << 60)) return -1;
    }
    return sum;
}

// The cache descriptor; fills the bytes that k and v span.
inline rope_status_t check_cache(const rope_kv_cache_t* c, int64_t* k_bytes, int64_t* v_bytes) {
    *k_bytes = *v_bytes = 0;
    if (!c) return fail(ROPE_ERR_NULLPTR, "cache is null");
    if (!valid_store(c->dtype))
        return fail(ROPE_ERR_INVALID, "cache dtype %d is not bf16 (0), fp16 (1), fp8 (3) or int8 (4)",
                    int(c->dtype));
    if (c->pages < 0 || c->page_size < 1 || c->heads < 1 || c->k_dim < 1 || c->v_dim < 0)
        return fail(ROPE_ERR_INVALID, "cache sizes: pages=%lld page_size=%lld heads=%lld k_dim=%lld "
                    "v_dim=%lld", (long long)c->pages, (long long)c->page_size,
                    (long long)c->heads, (long long)c->k_dim, (long long)c->v_dim);
    if (c->k_dim > 1024 || c->v_dim > 1024)
        return fail(ROPE_ERR_INVALID, "cache rows of %lld and %lld exceed 1024",
                    (long long)c->k_dim, (long long)c->v_dim);
    if (c->page_size > (int64_t(1) << 31) - 1 || c->pages > (int64_t(1) << 48) / c->page_size ||
        c->pages > kMaxSize || c->heads > (1 << 20))
        return fail(ROPE_ERR_INVALID, "cache sizes out of range");
    if (c->pages > 0 && !c->k) return fail(ROPE_ERR_NULLPTR, "cache k is null");
    if (c->pages > 0 && (c->v == nullptr) != (c->v_dim == 0))
        return fail(c->v ? ROPE_ERR_INVALID : ROPE_ERR_NULLPTR,
                    "cache v must be null exactly when v_dim is 0 (v_dim=%lld)", (long long)c->v_dim);
    const int e = code_size(c->dtype);
    const int64_t shape[3] = {c->pages, c->page_size, c->heads};
    const int64_t sk = span(shape, c->k_stride, 3, c->k_dim, c->k_dim);
    const int64_t sv = c->v_dim ? span(shape, c->v_stride, 3, c->v_dim, c->v_dim) : 0;
    if (sk < 0 || sv < 0)
        return fail(ROPE_ERR_INVALID, "cache strides must keep rows apart (at least the row length "
                    "on every dim of more than one)");
    if (!aligned(c->k, e) || !aligned(c->v, e))
        return fail(ROPE_ERR_INVALID, "cache k and v must be aligned to their %d-byte elements", e);
    if (e == 1) {
        if (c->pages > 0 && (!c->k_scale || (c->v_dim && !c->v_scale)))
            return fail(ROPE_ERR_NULLPTR, "an 8-bit cache needs k_scale and v_scale");
        if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
            return fail(ROPE_ERR_INVALID, "cache scales must be 4-byte aligned fp32");
        if (span(shape, c->k_scale_stride, 3, 1, 1) < 0 ||
            (c->v_dim && span(shape, c->v_scale_stride, 3, 1, 1) < 0))
            return fail(ROPE_ERR_INVALID, "cache scale strides must keep scales apart");
    } else if (c->k_scale || c->v_scale) {
        return fail(ROPE_ERR_INVALID, "a 16-bit cache has no scales");
    }
    *k_bytes = sk * e;
    *v_bytes = sv * e;
    return ROPE_OK;
}

// Whether [p, p + n) shares a byte with any part of the cache.
inline bool in_cache(const rope_kv_cache_t* c, int64_t kb, int64_t vb, const void* p, int64_t n) {
    if (c->pages == 0) return false;
    if (overlaps(p, n, c->k, kb) || (c->v && overlaps(p, n, c->v, vb))) return true;
    if (!c->k_scale) return false;
    const int64_t shape[3] = {c->pages, c->page_size, c->heads};
    return overlaps(p, n, c->k_scale, 4 * span(shape, c->k_scale_stride, 3, 1, 1)) ||
           (c->v_scale && overlaps(p, n, c->v_scale, 4 * span(shape, c->v_scale_stride, 3, 1, 1)));
}

// (The stride of a dim of one is not looked at by any call: 0 does for the kernels.)
inline int64_t step(int64_t size, int64_t stride) { return size > 1 ? stride : 0; }

// A tensor of (tokens, heads) rows: the bytes of a row, of a token's rows and of
// all, and the bytes between heads and between tokens (0: there is one).
struct Rows {
    const void* p;
    int64_t row, one, all, head, step;
};

inline Rows rows_of(const void* p, int64_t tokens, int64_t heads, const int64_t* stride, int64_t row, int e) {
    if (!p) return Rows{};
    const int64_t h = step(heads, stride[1]) * e, t = step(tokens, stride[0]) * e;
    const int64_t one = row * e + (heads - 1) * h;
    return Rows{p, row * e, one, one + (tokens - 1) * t, h, t};
}

// The bytes from a to the first of the places b + k * step that is not before it.
inline int64_t behind(const void* a, const void* b, int64_t step) {
    const uint64_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pb >= pa ? int64_t((pb - pa) % uint64_t(step)) : int64_t((step - int64_t((pa - pb) % uint64_t(step))) % step);
}

// Whether na bytes from 0 and nb bytes from `gap`, each repeated every `step`
// bytes, never meet.
inline bool apart(int64_t na, int64_t gap, int64_t nb, int64_t step) {
    return na <= step && nb <= step && gap % step >= na && gap % step + nb <= step;
}

// Whether two such tensors may share a byte.  Slices of one packed tensor
// (queries beside results, keys beside values) lie between each other.  With one
// step between tokens, they are apart when their bytes within it are.  With one
// step between heads also when their rows within that are, if a head of one token
// cannot meet a head of another: there is one token, the tokens' step is a multiple
// of the heads', or both tensors' tokens lie in the same steps.
inline bool rows_overlap(const Rows& a, const Rows& b) {
    if (!a.p || !b.p || !overlaps(a.p, a.all, b.p, b.all)) return false;
    if ((a.step && b.step && a.step != b.step) || (a.head && b.head && a.head != b.head)) return true;
    const int64_t step = a.step ? a.step : b.step, head = a.head ? a.head : b.head;
    const int64_t ab = step ? behind(a.p, b.p, step) : 0, ba = step ? behind(b.p, a.p, step) : 0;
    if (step && apart(a.one, ab, b.one, step)) return false;
    if (!head) return true;
    if (step == 0 || step % head == 0) return !apart(a.row, behind(a.p, b.p, head), b.row, head);
    if (a.one > step || b.one > step) return true;
    if (ab + b.one <= step) return !apart(a.row, ab, b.row, head);
    return ba + a.one > step || !apart(b.row, ba, a.row, head);
}

}  // namespace rope
