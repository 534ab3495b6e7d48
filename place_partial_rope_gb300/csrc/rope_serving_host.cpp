// rope_serving_host.cpp -- the C ABI entry points of include/rope_serving.h
// for the paged cache and the attention over it: argument checks, the choice
// of kernel and the launches.  No CUDA call is made for a rejected or empty
// call.
#include <float.h>
#include <math.h>
#include <string.h>

#include "rope_cache.h"
#include "rope_error.h"
#include "rope_tree.h"

namespace rope {
namespace {

constexpr int64_t kMaxSize = int64_t(1) << 40;  // of any one size or stride: products of two fit

int size_of(int dtype) { return dtype == ROPE_FP32 ? 4 : 2; }

bool valid_dtype(int d) { return d == ROPE_BF16 || d == ROPE_FP16 || d == ROPE_FP32; }

bool valid_store(int s) {
    return s == ROPE_CACHE_BF16 || s == ROPE_CACHE_FP16 || s == ROPE_CACHE_FP8 ||
           s == ROPE_CACHE_INT8;
}

int code_size(int store) { return store == ROPE_CACHE_BF16 || store == ROPE_CACHE_FP16 ? 2 : 1; }

bool aligned(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % uint64_t(n) == 0; }

// Elements from the first to the last of a tensor whose last dim (`row`
// elements) is contiguous; -1 when a stride is negative, or smaller than
// `apart` on a dim of more than one, or when the sum is out of range.
int64_t span(const int64_t* shape, const int64_t* stride, int n, int64_t row, int64_t apart) {
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
rope_status_t check_cache(const rope_kv_cache_t* c, int64_t* k_bytes, int64_t* v_bytes) {
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
bool in_cache(const rope_kv_cache_t* c, int64_t kb, int64_t vb, const void* p, int64_t n) {
    if (c->pages == 0) return false;
    if (overlaps(p, n, c->k, kb) || (c->v && overlaps(p, n, c->v, vb))) return true;
    if (!c->k_scale) return false;
    const int64_t shape[3] = {c->pages, c->page_size, c->heads};
    return overlaps(p, n, c->k_scale, 4 * span(shape, c->k_scale_stride, 3, 1, 1)) ||
           (c->v_scale && overlaps(p, n, c->v_scale, 4 * span(shape, c->v_scale_stride, 3, 1, 1)));
}

// (The stride of a dim of one is not looked at by any call: 0 does for the kernels.)
int64_t step(int64_t size, int64_t stride) { return size > 1 ? stride : 0; }

CacheSide side_of(const rope_kv_cache_t* c, bool values, void* rows, int64_t T, const int64_t* stride, int e) {
    const int ce = code_size(c->dtype);
    const int64_t* st = values ? c->v_stride : c->k_stride;
    const int64_t* ss = values ? c->v_scale_stride : c->k_scale_stride;
    CacheSide s{};
    s.rows = static_cast<char*>(rows);
    s.row_tok = step(T, stride[0]) * e;
    s.row_head = step(c->heads, stride[1]) * e;
    s.codes = static_cast<char*>(values ? c->v : c->k);
    s.page = step(c->pages, st[0]) * ce;
    s.tok = step(c->page_size, st[1]) * ce;
    s.head = step(c->heads, st[2]) * ce;
    s.scale = values ? c->v_scale : c->k_scale;
    s.s_page = ss[0];
    s.s_tok = ss[1];
    s.s_head = ss[2];
    s.dim = static_cast<int32_t>(values ? c->v_dim : c->k_dim);
    return s;
}

// Whether a side's rows allow accesses of n (8 or 16) elements.
bool wide(const rope_kv_cache_t* c, const CacheSide& s, int n) {
    const int64_t ce = n * code_size(c->dtype);
    bool ok = s.dim % n == 0 && aligned(s.rows, 16) && aligned(s.codes, ce);
    const int64_t dense[2] = {s.row_tok, s.row_head}, codes[3] = {s.page, s.tok, s.head};
    for (int64_t v : dense) ok = ok && v % 16 == 0;
    for (int64_t v : codes) ok = ok && v % ce == 0;
    return ok;
}

// A tensor of (tokens, heads) rows: the bytes of a row, of a token's rows and of
// all, and the bytes between heads and between tokens (0: there is one).
struct Rows {
    const void* p;
    int64_t row, one, all, head, step;
};

Rows rows_of(const void* p, int64_t tokens, int64_t heads, const int64_t* stride, int64_t row, int e) {
    if (!p) return Rows{};
    const int64_t h = step(heads, stride[1]) * e, t = step(tokens, stride[0]) * e;
    const int64_t one = row * e + (heads - 1) * h;
    return Rows{p, row * e, one, one + (tokens - 1) * t, h, t};
}

// The bytes from a to the first of the places b + k * step that is not before it.
int64_t behind(const void* a, const void* b, int64_t step) {
    const uint64_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pb >= pa ? int64_t((pb - pa) % uint64_t(step)) : int64_t((step - int64_t((pa - pb) % uint64_t(step))) % step);
}

// Whether na bytes from 0 and nb bytes from `gap`, each repeated every `step`
// bytes, never meet.
bool apart(int64_t na, int64_t gap, int64_t nb, int64_t step) {
    return na <= step && nb <= step && gap % step >= na && gap % step + nb <= step;
}

// Whether two such tensors may share a byte.  Slices of one packed tensor
// (queries beside results, keys beside values) lie between each other.  With one
// step between tokens, they are apart when their bytes within it are.  With one
// step between heads also when their rows within that are, if a head of one token
// cannot meet a head of another: there is one token, the tokens' step is a multiple
// of the heads', or both tensors' tokens lie in the same steps.
bool rows_overlap(const Rows& a, const Rows& b) {
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

// What write and read have in common: T rows a token, split into launches
// whose row index fits 32 bits.
template <typename Launch>
rope_status_t run_rows(const rope_kv_cache_t* c, CachePlan plan, CacheArgs a, bool keys, bool values,
                       bool write, int64_t T, Launch&& go) {
    int64_t dim = 0;
    bool w = true, w16 = !write && code_size(c->dtype) == 1;
    for (int i = 0; i < 2; ++i) {
        if (!(i ? values : keys)) continue;
        if (a.side[i].dim > dim) dim = a.side[i].dim;
        w = w && wide(c, a.side[i], 8);
        w16 = w16 && wide(c, a.side[i], 16);
    }
    if (w16 && dim <= 256) plan.vec = 16, plan.lanes = 4;
    else if (w) plan.vec = 8, plan.lanes = dim <= 256 ? 8 : 32;
    else plan.vec = 1, plan.lanes = 32;
    plan.chunks = static_cast<int>((dim + plan.vec * plan.lanes - 1) / (plan.vec * plan.lanes));
    if (!w) plan.turn = false;
    a.total = uint64_t(c->pages) * uint64_t(c->page_size);
    a.page_size = c->page_size;
    a.div_page = FastDiv::make(static_cast<uint32_t>(c->page_size));
    a.heads = static_cast<int32_t>(c->heads);
    a.first = keys ? 0 : 1;
    const int64_t per = c->heads * (keys && values ? 2 : 1);
    a.div_rows = FastDiv::make(static_cast<uint32_t>(per));
    const int64_t most = (int64_t(1) << 31) / per;  // tokens of one launch
    for (int64_t t = 0; t < T; t += most) {
        const int64_t n = T - t < most ? T - t : most;
        CacheArgs p = a;
        p.rows = static_cast<uint32_t>(n * per);
        p.slots += t;
        for (CacheSide& s : p.side)
            if (s.rows) s.rows += t * s.row_tok;
        if (p.cos) p.cos += t * p.cos_tok;
        if (p.sin) p.sin += t * p.sin_tok;
        const char* err = nullptr;
        if (go(plan, p, &err) != ROPE_OK) return fail(ROPE_ERR_CUDA, "%s", err);
    }
    return ROPE_OK;
}

rope_status_t cache_write(const rope_kv_cache_t* c, const void* k, const void* v, int dtype,
                          int64_t T, const int64_t* k_stride, const int64_t* v_stride,
                          const int64_t* slots, const void* cos, const void* sin,
                          int64_t cos_stride, int64_t sin_stride, int64_t start, int64_t end,
                          int mode, rope_stream_t stream) {
    clear_error();
    int64_t kb, vb;
    rope_status_t st = check_cache(c, &kb, &vb);
    if (st != ROPE_OK) return st;
    if (!valid_dtype(dtype))
        return fail(ROPE_ERR_INVALID, "dtype %d is not bf16 (0), fp16 (1) or fp32 (2)", dtype);
    if (mode != ROPE_MODE_INTERLEAVE && mode != ROPE_MODE_HALF)
        return fail(ROPE_ERR_INVALID, "rotary mode %d is not interleave (1) or half (2)", mode);
    if (T < 0 || T > kMaxSize) return fail(ROPE_ERR_INVALID, "T=%lld tokens", (long long)T);
    if (start < 0 || end < start || end > c->k_dim)
        return fail(ROPE_ERR_INVALID, "partial slice [%lld, %lld) must satisfy 0 <= start <= end <= "
                    "k_dim=%lld", (long long)start, (long long)end, (long long)c->k_dim);
    const int64_t L = end - start;
    if (L % 2 != 0)
        return fail(ROPE_ERR_INVALID, "slice length end - start = %lld must be even", (long long)L);
    if (T == 0) return ROPE_OK;
    if (!k || !slots || !k_stride) return fail(ROPE_ERR_NULLPTR, "k, its strides or slots is null");
    if ((v == nullptr) != (c->v_dim == 0))
        return fail(v ? ROPE_ERR_INVALID : ROPE_ERR_NULLPTR,
                    "v must be null exactly when the cache has no values");
    if (v && !v_stride) return fail(ROPE_ERR_NULLPTR, "v_stride is null");
    if (L > 0 && (!cos || !sin)) return fail(ROPE_ERR_NULLPTR, "cos or sin is null");
    const int e = size_of(dtype);
    const int64_t shape[2] = {T, c->heads};
    const int64_t sk = span(shape, k_stride, 2, c->k_dim, 0);
    const int64_t sv = v ? span(shape, v_stride, 2, c->v_dim, 0) : 0;
    const int64_t sc = L ? span(shape, &cos_stride, 1, L, 0) : 0;
    const int64_t ss = L ? span(shape, &sin_stride, 1, L, 0) : 0;
    if (sk < 0 || sv < 0 || sc < 0 || ss < 0)
        return fail(ROPE_ERR_INVALID, "strides of k, v, cos and sin must be >= 0 and in range");
    if (!aligned(k, e) || !aligned(v, e) || (L && (!aligned(cos, e) || !aligned(sin, e))) ||
        !aligned(slots, 8))
        return fail(ROPE_ERR_INVALID, "k, v, cos, sin and slots must be aligned to their elements");
    if (in_cache(c, kb, vb, k, sk * e) || (v && in_cache(c, kb, vb, v, sv * e)) ||
        in_cache(c, kb, vb, slots, 8 * T) ||
        (L && (in_cache(c, kb, vb, cos, sc * e) || in_cache(c, kb, vb, sin, ss * e))))
        return fail(ROPE_ERR_INVALID, "an input overlaps the cache, which is written");
    if (c->pages == 0) return ROPE_OK;  // every slot lies outside

    CacheArgs a{};
    a.side[0] = side_of(c, false, const_cast<void*>(k), T, k_stride, e);
    if (v) a.side[1] = side_of(c, true, const_cast<void*>(v), T, v_stride, e);
    a.slots = slots;
    a.start = static_cast<int32_t>(start);
    a.half = static_cast<int32_t>(L / 2);
    a.half_mode = mode == ROPE_MODE_HALF;
    CachePlan plan{};
    plan.dtype = dtype;
    plan.store = c->dtype;
    if (L) {
        a.cos = static_cast<const char*>(cos);
        a.sin = static_cast<const char*>(sin);
        a.cos_tok = step(T, cos_stride) * e;
        a.sin_tok = step(T, sin_stride) * e;
        // 8-element accesses that lie wholly inside or outside the slice,
        // and whose half-split partners are whole accesses too
        plan.turn = start % 8 == 0 && (a.half_mode ? (L / 2) % 8 == 0 : L % 8 == 0) &&
                    aligned(cos, 16) && aligned(sin, 16) && a.cos_tok % 16 == 0 &&
                    a.sin_tok % 16 == 0;
    } else {
        plan.turn = true;  // nothing turns: either instance will do
    }
    return run_rows(c, plan, a, true, v != nullptr, true, T,
                    [&](const CachePlan& p, const CacheArgs& q, const char** err) {
                        return launch_cache_write(p, q, stream, err);
                    });
}

rope_status_t cache_read(const rope_kv_cache_t* c, const int64_t* slots, int64_t T, void* k, void* v,
                         int dtype, const int64_t* k_stride, const int64_t* v_stride,
                         rope_stream_t stream) {
    clear_error();
    int64_t kb, vb;
    rope_status_t st = check_cache(c, &kb, &vb);
    if (st != ROPE_OK) return st;
    if (!valid_dtype(dtype))
        return fail(ROPE_ERR_INVALID, "dtype %d is not bf16 (0), fp16 (1) or fp32 (2)", dtype);
    if (T < 0 || T > kMaxSize) return fail(ROPE_ERR_INVALID, "T=%lld tokens", (long long)T);
    if (v && c->v_dim == 0) return fail(ROPE_ERR_INVALID, "the cache has no values");
    if (T == 0 || (!k && !v)) return ROPE_OK;
    if (!slots) return fail(ROPE_ERR_NULLPTR, "slots is null");
    if ((k && !k_stride) || (v && !v_stride)) return fail(ROPE_ERR_NULLPTR, "k_stride or v_stride is null");
    const int e = size_of(dtype);
    const int64_t shape[2] = {T, c->heads};
    const int64_t sk = k ? span(shape, k_stride, 2, c->k_dim, c->k_dim) : 0;
    const int64_t sv = v ? span(shape, v_stride, 2, c->v_dim, c->v_dim) : 0;
    if (sk < 0 || sv < 0)
        return fail(ROPE_ERR_INVALID, "strides of k and v must keep rows apart and be in range");
    if (!aligned(k, e) || !aligned(v, e) || !aligned(slots, 8))
        return fail(ROPE_ERR_INVALID, "k, v and slots must be aligned to their elements");
    const Rows kr = rows_of(k, T, c->heads, k_stride, c->k_dim, e);
    const Rows vr = rows_of(v, T, c->heads, v_stride, c->v_dim, e);
    if (rows_overlap(kr, vr) || overlaps(k, sk * e, slots, 8 * T) ||
        overlaps(v, sv * e, slots, 8 * T) || in_cache(c, kb, vb, k, sk * e) ||
        in_cache(c, kb, vb, v, sv * e))
        return fail(ROPE_ERR_INVALID, "the outputs overlap each other, the slots or the cache");

    CacheArgs a{};
    if (k) a.side[0] = side_of(c, false, k, T, k_stride, e);
    if (v) a.side[1] = side_of(c, true, v, T, v_stride, e);
    a.slots = slots;
    CachePlan plan{};
    plan.dtype = dtype;
    plan.store = c->dtype;
    return run_rows(c, plan, a, k != nullptr, v != nullptr, false, T,
                    [&](const CachePlan& p, const CacheArgs& q, const char** err) {
                        return launch_cache_read(p, q, stream, err);
                    });
}

// ------------------------------------------------------------------------
// attention
// ------------------------------------------------------------------------

// What the kernel choice depends on: types, row lengths, the query rows that
// share a key head, and the cache tiles (of 128 rows) that there can be.
rope_status_t tree_plan(const rope_kv_cache_t* c, int dtype, int64_t Hq, int64_t max_q, int64_t tiles,
                        TreePlan* p) {
    if (dtype != ROPE_BF16 && dtype != ROPE_FP16)
        return fail(ROPE_ERR_INVALID, "attention takes bf16 (0) or fp16 (1), not dtype %d", dtype);
    if (code_size(c->dtype) == 2 && c->dtype != dtype)
        return fail(ROPE_ERR_INVALID, "a 16-bit cache must have the type of q (cache %d, q %d)",
                    int(c->dtype), dtype);
    if (c->k_dim > 256 || c->v_dim > c->k_dim || c->v_dim < 16 || c->k_dim % 16 || c->v_dim % 16)
        return fail(ROPE_ERR_INVALID, "k_dim=%lld and v_dim=%lld must be multiples of 16 with 16 <= "
                    "v_dim <= k_dim <= 256", (long long)c->k_dim, (long long)c->v_dim);
    if (Hq < 1 || Hq > (1 << 20) || Hq % c->heads)
        return fail(ROPE_ERR_INVALID, "Hq=%lld must be a multiple of the cache's %lld heads",
                    (long long)Hq, (long long)c->heads);
    if (max_q < 1 || max_q > (int64_t(1) << 31) - 1)
        return fail(ROPE_ERR_INVALID, "max_q=%lld must be positive", (long long)max_q);
    p->dtype = dtype;
    p->store = c->dtype;
    choose_tree(static_cast<int>(c->k_dim), static_cast<int>(c->v_dim), max_q * (Hq / c->heads),
                c->pages, c->page_size, tiles, p);
    return ROPE_OK;
}

rope_status_t tree_attention(const rope_kv_cache_t* c, const void* q, int dtype, int64_t Tq,
                             int64_t Hq, const int64_t* q_stride, const int32_t* q_start,
                             const int32_t* kv_len, int64_t R, int64_t max_q,
                             const int32_t* page_table, int64_t max_pages, int64_t table_stride,
                             const int64_t* tree, int64_t words, void* out,
                             const int64_t* out_stride, float* lse, double scale, void* workspace,
                             int64_t workspace_bytes, rope_stream_t stream) {
    clear_error();
    int64_t kb, vb;
    rope_status_t st = check_cache(c, &kb, &vb);
    if (st != ROPE_OK) return st;
    constexpr int64_t kInt = (int64_t(1) << 31) - 1;
    // (sizes that overflow here are refused below)
    const double room = double(R) * double(c->heads) * (double(max_pages) * double(c->page_size) / 128.0 + 1.0);
    TreePlan p{};
    st = tree_plan(c, dtype, Hq, max_q, room < 1e15 ? static_cast<int64_t>(room) : kInt, &p);
    if (st != ROPE_OK) return st;
    if (Tq < 0 || Tq > kInt / Hq || R < 0 || R > (1 << 24))
        return fail(ROPE_ERR_INVALID, "Tq=%lld query tokens, R=%lld requests", (long long)Tq,
                    (long long)R);
    if (max_pages < 0 || max_pages > kInt || max_pages * c->page_size > kInt - 1024)
        return fail(ROPE_ERR_INVALID, "%lld pages of %lld tokens a request exceed 2^31 rows",
                    (long long)max_pages, (long long)c->page_size);
    if (c->pages > kInt) return fail(ROPE_ERR_INVALID, "more than 2^31 pages");
    if (table_stride < 0 || (R > 1 && table_stride < max_pages) || table_stride > kMaxSize)
        return fail(ROPE_ERR_INVALID, "page_table_stride %lld is less than max_pages %lld",
                    (long long)table_stride, (long long)max_pages);
    if (tree && (words < 1 || words > kInt / 64))
        return fail(ROPE_ERR_INVALID, "tree_words=%lld must be positive", (long long)words);
    const float scale_log2 = static_cast<float>(scale * 1.4426950408889634);
    if (!(scale > 0.0) || !isfinite(scale_log2) || scale_log2 < FLT_MIN)
        return fail(ROPE_ERR_INVALID, "scale %g must be a number > 0 that fp32 holds (times log2(e))", scale);
    if (Tq == 0 || R == 0) return ROPE_OK;
    if (!q || !out || !q_stride || !out_stride || !q_start || !kv_len)
        return fail(ROPE_ERR_NULLPTR, "q, out, their strides, q_start or kv_len is null");
    if (!page_table && max_pages > 0) return fail(ROPE_ERR_NULLPTR, "page_table is null");
    if (!workspace) return fail(ROPE_ERR_NULLPTR, "workspace is null");
    const int ce = code_size(c->dtype);
    const int64_t shape[2] = {Tq, Hq};
    const int64_t sq = span(shape, q_stride, 2, c->k_dim, 0);
    const int64_t so = span(shape, out_stride, 2, c->v_dim, c->v_dim);
    if (sq < 0 || so < 0)
        return fail(ROPE_ERR_INVALID, "strides of q and out must be >= 0, and keep the rows of out apart");
    bool ok = aligned(q, 16) && aligned(out, 16) && aligned(c->k, 16) && aligned(c->v, 16) &&
              aligned(workspace, 16);
    const int64_t slots[3] = {c->pages, c->page_size, c->heads};
    for (int i = 0; i < 2; ++i)
        ok = ok && step(shape[i], q_stride[i]) * 2 % 16 == 0 && step(shape[i], out_stride[i]) * 2 % 16 == 0;
    for (int i = 0; i < 3; ++i)
        ok = ok && step(slots[i], c->k_stride[i]) * ce % 16 == 0 && step(slots[i], c->v_stride[i]) * ce % 16 == 0;
    if (!ok)
        return fail(ROPE_ERR_INVALID, "the rows of q, out and the cache and the workspace must start "
                    "on 16-byte boundaries");
    if (!aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4) || !aligned(tree, 8) ||
        !aligned(lse, 4))
        return fail(ROPE_ERR_INVALID, "q_start, kv_len, page_table, tree and lse must be aligned to "
                    "their elements");
    // out, lse and the workspace are written while everything else is read
    const struct { const void* p; int64_t n; } wr[3] = {
        {out, so * 2}, {lse, lse ? Tq * Hq * 4 : 0}, {workspace, workspace_bytes}};
    const struct { const void* p; int64_t n; } rd[4] = {
        {q_start, (R + 1) * 4}, {kv_len, R * 4},
        {page_table, max_pages ? ((R - 1) * table_stride + max_pages) * 4 : 0},
        {tree, tree ? Tq * words * 8 : 0}};
    const Rows qr = rows_of(q, Tq, Hq, q_stride, c->k_dim, 2);
    const Rows outr = rows_of(out, Tq, Hq, out_stride, c->v_dim, 2);
    bool shared = rows_overlap(qr, outr) || overlaps(q, sq * 2, wr[1].p, wr[1].n) ||
                  overlaps(q, sq * 2, wr[2].p, wr[2].n);
    for (int i = 0; i < 3; ++i) {
        bool hit = shared || in_cache(c, kb, vb, wr[i].p, wr[i].n);
        for (const auto& r : rd) hit = hit || overlaps(wr[i].p, wr[i].n, r.p, r.n);
        for (int j = 0; j < i; ++j) hit = hit || overlaps(wr[i].p, wr[i].n, wr[j].p, wr[j].n);
        if (hit) return fail(ROPE_ERR_INVALID, "out, lse and workspace must not overlap each other or "
                             "anything that is read");
    }

    const char* err = nullptr;
    int blocks = 0;
    if (tree_blocks(p, 0, &blocks, &err) != ROPE_OK) return fail(ROPE_ERR_CUDA, "%s", err);
    const int64_t need = tree_workspace(p, blocks);
    if (workspace_bytes < need)
        return fail(ROPE_ERR_INVALID, "workspace of %lld bytes; the call needs %lld",
                    (long long)workspace_bytes, (long long)need);

    TreeArgs a{};
    // (no pages: no row is read, but the kernel forms an address all the same)
    a.k = static_cast<const char*>(c->pages ? c->k : q);
    a.v = static_cast<const char*>(c->pages ? c->v : q);
    a.ks = c->pages ? c->k_scale : static_cast<const float*>(q);
    a.vs = c->pages ? c->v_scale : static_cast<const float*>(q);
    for (int i = 0; i < 3; ++i) {
        a.k_st[i] = step(slots[i], c->k_stride[i]) * ce;
        a.v_st[i] = step(slots[i], c->v_stride[i]) * ce;
        a.ks_st[i] = c->k_scale_stride[i];
        a.vs_st[i] = c->v_scale_stride[i];
    }
    a.q = static_cast<const char*>(q);
    a.out = static_cast<char*>(out);
    a.lse = lse;
    for (int i = 0; i < 2; ++i) {
        a.q_st[i] = step(shape[i], q_stride[i]) * 2;
        a.o_st[i] = step(shape[i], out_stride[i]) * 2;
    }
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.table = page_table;
    a.table_stride = table_stride;
    a.tree = tree;
    a.words = static_cast<int32_t>(tree ? words : 0);
    a.R = static_cast<int32_t>(R);
    a.Tq = static_cast<int32_t>(Tq);
    a.Hk = static_cast<int32_t>(c->heads);
    a.G = static_cast<int32_t>(Hq / c->heads);
    a.Hq = static_cast<int32_t>(Hq);
    a.Dk = static_cast<int32_t>(c->k_dim);
    a.Dv = static_cast<int32_t>(c->v_dim);
    a.pages = static_cast<int32_t>(c->pages);
    a.page_size = static_cast<int32_t>(c->page_size);
    a.max_len = static_cast<int32_t>(max_pages * c->page_size);
    a.div_page = FastDiv::make(static_cast<uint32_t>(c->page_size));
    a.div_group = FastDiv::make(static_cast<uint32_t>(Hq / c->heads));
    a.scale_log2 = scale_log2;
    a.bf16 = dtype == ROPE_BF16;
    if (launch_tree(p, a, workspace, blocks, stream, &err) != ROPE_OK)
        return fail(ROPE_ERR_CUDA, "%s", err);
    return ROPE_OK;
}

}  // namespace
}  // namespace rope

extern "C" {

rope_status_t rope_partial_cache_write(const rope_kv_cache_t* cache, const void* k, const void* v,
                                       rope_dtype_t dtype, int64_t T, const int64_t k_stride[2],
                                       const int64_t v_stride[2], const int64_t* slots,
                                       const void* cos, const void* sin, int64_t cos_stride,
                                       int64_t sin_stride, int64_t start, int64_t end,
                                       rope_mode_t mode, rope_stream_t stream) {
    return rope::cache_write(cache, k, v, static_cast<int>(dtype), T, k_stride, v_stride, slots, cos,
                             sin, cos_stride, sin_stride, start, end, static_cast<int>(mode), stream);
}

rope_status_t rope_partial_cache_read(const rope_kv_cache_t* cache, const int64_t* slots, int64_t T,
                                      void* k, void* v, rope_dtype_t dtype,
                                      const int64_t k_stride[2], const int64_t v_stride[2],
                                      rope_stream_t stream) {
    return rope::cache_read(cache, slots, T, k, v, static_cast<int>(dtype), k_stride, v_stride, stream);
}

rope_status_t rope_partial_tree_attention(const rope_kv_cache_t* cache, const void* q,
                                          rope_dtype_t dtype, int64_t Tq, int64_t Hq,
                                          const int64_t q_stride[2], const int32_t* q_start,
                                          const int32_t* kv_len, int64_t R, int64_t max_q,
                                          const int32_t* page_table, int64_t max_pages,
                                          int64_t page_table_stride, const int64_t* tree,
                                          int64_t tree_words, void* out,
                                          const int64_t out_stride[2], float* lse, double scale,
                                          void* workspace, int64_t workspace_bytes,
                                          rope_stream_t stream) {
    return rope::tree_attention(cache, q, static_cast<int>(dtype), Tq, Hq, q_stride, q_start, kv_len,
                                R, max_q, page_table, max_pages, page_table_stride, tree, tree_words,
                                out, out_stride, lse, scale, workspace, workspace_bytes, stream);
}

rope_status_t rope_partial_tree_attention_workspace(const rope_kv_cache_t* cache,
                                                    rope_dtype_t dtype, int64_t Hq, int64_t max_q,
                                                    int32_t sm_count, int64_t* bytes) {
    using namespace rope;
    clear_error();
    if (!bytes) return fail(ROPE_ERR_NULLPTR, "bytes is null");
    if (sm_count < 0) return fail(ROPE_ERR_INVALID, "sm_count is negative");
    int64_t kb, vb;
    rope_status_t st = check_cache(cache, &kb, &vb);
    if (st != ROPE_OK) return st;
    int64_t most = 0;
    for (int many = 0; many < 2; ++many) {  // a call of few cache tiles, and of many
        TreePlan p{};
        st = tree_plan(cache, static_cast<int>(dtype), Hq, max_q, many ? int64_t(1) << 31 : 0, &p);
        if (st != ROPE_OK) return st;
        const char* err = nullptr;
        int blocks = 0;
        if (tree_blocks(p, sm_count, &blocks, &err) != ROPE_OK) return fail(ROPE_ERR_CUDA, "%s", err);
        const int64_t need = tree_workspace(p, blocks);
        if (need > most) most = need;
    }
    *bytes = most;
    return ROPE_OK;
}

rope_status_t rope_partial_tree_mask(const int32_t* parents, int64_t n, int64_t tree_words,
                                     int64_t* words) {
    using namespace rope;
    clear_error();
    if (n < 0 || tree_words < 0 || tree_words < (n + 63) / 64)
        return fail(ROPE_ERR_INVALID, "%lld drafted tokens do not fit %lld words", (long long)n,
                    (long long)tree_words);
    if (n == 0) return ROPE_OK;
    if (!parents || !words) return fail(ROPE_ERR_NULLPTR, "parents or words is null");
    for (int64_t i = 0; i < n; ++i)
        if (parents[i] < -1 || parents[i] >= i)
            return fail(ROPE_ERR_INVALID, "parent %lld is %d; it must be -1 or an earlier token",
                        (long long)i, int(parents[i]));
    for (int64_t i = 0; i < n; ++i) {
        int64_t* row = words + i * tree_words;
        if (parents[i] < 0) memset(row, 0, sizeof(int64_t) * tree_words);
        else memcpy(row, words + parents[i] * tree_words, sizeof(int64_t) * tree_words);
        row[i / 64] = static_cast<int64_t>(static_cast<uint64_t>(row[i / 64]) | uint64_t(1) << (i % 64));
    }
    return ROPE_OK;
}

}  // extern "C"
