// rope_norm_host.cpp -- the C ABI entry points of include/rope_step.h for the norm
// and rotation: argument checks, the choice of kernel and the launches.  No
// CUDA call is made for a rejected call, or a forward of no rows.
#include <math.h>

#include "rope_check.h"
#include "rope_norm.h"

namespace rope {
namespace {

// A (B, S, heads) tensor of rows; strides in elements.
struct Tensor {
    const void* p;
    const int64_t* shape;
    const int64_t* stride;
    int64_t row;  // elements
    int e;        // bytes of one

    int64_t at(int i) const { return step(shape[i], stride[i]) * e; }
    // bytes from the first to the last
    int64_t all() const { return span(shape, stride, 3, row, 0) * e; }
};

// Whether the rows of a tensor are apart from each other: each stride steps over
// all that the smaller ones span.
bool rows_apart(const Tensor& t) {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (t.at(order[j]) < t.at(order[i])) {
                const int x = order[i];
                order[i] = order[j];
                order[j] = x;
            }
    int64_t extent = t.row * t.e;
    for (int i : order) {
        if (t.shape[i] <= 1) continue;
        if (t.at(i) < extent) return false;
        extent += (t.shape[i] - 1) * t.at(i);
    }
    return true;
}

// Whether two tensors of the same batches and tokens may share a byte.  Heads of one
// projection's rows lie between each other (rows_overlap).  Batches count as one
// more run of tokens where they follow each other, or apart from each other where both
// tensors' lie in the same steps.
bool tensors_overlap(const Tensor& a, const Tensor& b) {
    if (!overlaps(a.p, a.all(), b.p, b.all())) return false;
    const int64_t B = a.shape[0], S = a.shape[1];
    int64_t tokens = B * S, sa = a.at(1), sb = b.at(1);
    if (S == 1) {
        sa = a.at(0), sb = b.at(0);
    } else if (B > 1 && (a.at(0) != S * sa || b.at(0) != S * sb)) {
        const int64_t step = a.at(0);
        if (b.at(0) != step) return true;
        const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
        const int64_t one[3] = {1, S, 0};
        const int64_t ha[3] = {one[0], S, a.shape[2]}, hb[3] = {one[0], S, b.shape[2]};
        const Tensor x{a.p, ha, a.stride, a.row, a.e}, y{b.p, hb, b.stride, b.row, b.e};
        const uintptr_t lo = pa < pb ? pa : pb;
        const uintptr_t ea = pa + uintptr_t(x.all()), eb = pb + uintptr_t(y.all());
        if (int64_t((ea > eb ? ea : eb) - lo) > step) return true;
        tokens = S;
    }
    auto rows = [&](const Tensor& t, int64_t s) {
        const int64_t h = t.at(2), one = t.row * t.e + (t.shape[2] - 1) * h;
        return Rows{t.p, t.row * t.e, one, one + (tokens - 1) * s, h, tokens > 1 ? s : 0};
    };
    return rows_overlap(rows(a, sa), rows(b, sb));
}

bool same(const Tensor& a, const Tensor& b) {
    if (a.p != b.p) return false;
    for (int i = 0; i < 3; ++i)
        if (a.at(i) != b.at(i)) return false;
    return true;
}

struct Call {
    int dtype, weight_dtype;
    int64_t B, S, D, n0, n1;
    double eps;
    const void *cos, *sin;
    const int64_t *cos_stride, *sin_stride;
    int64_t start, end;
    int mode;
    bool back;
    void* workspace;
    int64_t workspace_bytes;
};

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

// What is read or written besides the rows: byte ranges.
struct Range {
    const void* p;
    int64_t n;
};

rope_status_t check_side(const rope_norm_rows_t* r, const char* name, const Call& c) {
    const int e = size_of(c.dtype);
    if (r->heads < 1 || r->heads > (1 << 20))
        return fail(ROPE_ERR_INVALID, "%s: heads=%lld must be positive", name, (long long)r->heads);
    if (c.B * c.S > kMaxRows / r->heads)  // (both below 2^31 by now)
        return fail(ROPE_ERR_INVALID, "%s: 2^31 rows or more", name);
    // (written also where there are no rows)
    if (c.back && !aligned(r->weight_grad, 4))
        return fail(ROPE_ERR_INVALID, "%s: weight_grad must be aligned to its elements", name);
    if (c.B * c.S == 0) return ROPE_OK;
    if (!r->x || !r->out || (c.back && (!r->grad || !r->rstd)))
        return fail(ROPE_ERR_NULLPTR, "%s: x, out%s is null", name, c.back ? ", grad or rstd" : "");
    const int64_t shape[3] = {c.B, c.S, r->heads};
    const Tensor x{r->x, shape, r->x_stride, c.D, e}, out{r->out, shape, r->out_stride, c.D, e},
        grad{r->grad, shape, r->grad_stride, c.D, e};
    if (x.all() < 0 || out.all() < 0 || (c.back && grad.all() < 0))
        return fail(ROPE_ERR_INVALID, "%s: strides must be >= 0 and in range", name);
    if (!rows_apart(out)) return fail(ROPE_ERR_INVALID, "%s: strides of out must keep its rows apart", name);
    if (!aligned(r->x, e) || !aligned(r->out, e) || (c.back && !aligned(r->grad, e)) || !aligned(r->rstd, 4) ||
        !aligned(r->weight, size_of(c.weight_dtype)))
        return fail(ROPE_ERR_INVALID, "%s: pointers must be aligned to their elements", name);
    return ROPE_OK;
}

// Outputs share no byte with anything, but for out with x (backward: grad) as a whole.
rope_status_t check_overlap(const rope_norm_rows_t* const* sides, int n, const Call& c) {
    const int e = size_of(c.dtype);
    const int64_t normed = c.n1 - c.n0;
    Tensor read[4], written[2];
    int64_t shape[2][3];
    Range in[6], out[5];
    int reads = 0, ins = 0, outs = 0;
    for (int i = 0; i < n; ++i) {
        const rope_norm_rows_t* r = sides[i];
        shape[i][0] = c.B, shape[i][1] = c.S, shape[i][2] = r->heads;
        read[reads++] = Tensor{r->x, shape[i], r->x_stride, c.D, e};
        if (c.back) read[reads++] = Tensor{r->grad, shape[i], r->grad_stride, c.D, e};
        written[i] = Tensor{r->out, shape[i], r->out_stride, c.D, e};
        const Range rstd{r->rstd, r->rstd ? c.B * c.S * r->heads * 4 : 0};
        (c.back ? in[ins++] : out[outs++]) = rstd;
        in[ins++] = Range{r->weight, r->weight ? normed * size_of(c.weight_dtype) : 0};
        if (c.back) out[outs++] = Range{r->weight_grad, r->weight_grad ? normed * 4 : 0};
    }
    if (c.back) out[outs++] = Range{c.workspace, c.workspace ? c.workspace_bytes : 0};
    const int64_t L = c.end - c.start, tokens[2] = {c.B, c.S};
    if (L) {
        in[ins++] = Range{c.cos, span(tokens, c.cos_stride, 2, L, 0) * e};
        in[ins++] = Range{c.sin, span(tokens, c.sin_stride, 2, L, 0) * e};
    }
    bool hit = false;
    for (int i = 0; i < n; ++i) {
        const Tensor& own = read[c.back ? 2 * i + 1 : i];  // what out may be
        for (int j = 0; j < reads; ++j)
            if (!(&read[j] == &own && same(own, written[i]))) hit = hit || tensors_overlap(written[i], read[j]);
        for (int j = 0; j < i; ++j) hit = hit || tensors_overlap(written[i], written[j]);
        for (int j = 0; j < ins; ++j) hit = hit || overlaps(written[i].p, written[i].all(), in[j].p, in[j].n);
        for (int j = 0; j < outs; ++j) hit = hit || overlaps(written[i].p, written[i].all(), out[j].p, out[j].n);
    }
    for (int i = 0; i < outs; ++i) {
        for (int j = 0; j < reads; ++j) hit = hit || overlaps(out[i].p, out[i].n, read[j].p, read[j].all());
        for (int j = 0; j < ins; ++j) hit = hit || overlaps(out[i].p, out[i].n, in[j].p, in[j].n);
        for (int j = 0; j < i; ++j) hit = hit || overlaps(out[i].p, out[i].n, out[j].p, out[j].n);
    }
    if (hit)
        return fail(ROPE_ERR_INVALID, "an output overlaps another or what is read (out may be %s as a whole)",
                    c.back ? "grad" : "x");
    return ROPE_OK;
}

rope_status_t norm_workspace(int64_t normed, int sms, int64_t* bytes) {
    *bytes = normed * sms * kNormBlocksPerSm * 2 * int64_t(sizeof(float));
    return ROPE_OK;
}

rope_status_t norm(const rope_norm_rows_t* q, const rope_norm_rows_t* k, const Call& c, rope_stream_t stream) {
    clear_error();
    if (!q) return fail(ROPE_ERR_NULLPTR, "q is null");
    if (!valid_dtype(c.dtype))
        return fail(ROPE_ERR_INVALID, "dtype %d is not bf16 (0), fp16 (1) or fp32 (2)", c.dtype);
    if (c.weight_dtype != c.dtype && c.weight_dtype != ROPE_FP32)
        return fail(ROPE_ERR_INVALID, "weight_dtype %d is neither dtype (%d) nor fp32 (2)", c.weight_dtype, c.dtype);
    if (c.mode != ROPE_MODE_INTERLEAVE && c.mode != ROPE_MODE_HALF)
        return fail(ROPE_ERR_INVALID, "rotary mode %d is not interleave (1) or half (2)", c.mode);
    if (c.B < 0 || c.S < 0 || c.B > kMaxRows || c.S > kMaxRows)
        return fail(ROPE_ERR_INVALID, "sizes: B=%lld S=%lld", (long long)c.B, (long long)c.S);
    if (c.D < 1 || c.D > 1024) return fail(ROPE_ERR_INVALID, "D=%lld must be 1 .. 1024", (long long)c.D);
    if (c.n0 < 0 || c.n1 <= c.n0 || c.n1 > c.D)
        return fail(ROPE_ERR_INVALID, "normed lanes [%lld, %lld) must satisfy 0 <= norm_start < norm_end <= D=%lld",
                    (long long)c.n0, (long long)c.n1, (long long)c.D);
    if (!(c.eps >= 0.0) || !isfinite(static_cast<float>(c.eps)))
        return fail(ROPE_ERR_INVALID, "eps %g must be a number >= 0 that fp32 holds", c.eps);
    if (c.start < 0 || c.end < c.start || c.end > c.D)
        return fail(ROPE_ERR_INVALID, "partial slice [%lld, %lld) must satisfy 0 <= start <= end <= D=%lld",
                    (long long)c.start, (long long)c.end, (long long)c.D);
    const int64_t L = c.end - c.start;
    if (L % 2 != 0)
        return fail(ROPE_ERR_INVALID, "slice length end - start = %lld must be even", (long long)L);
    const rope_norm_rows_t* sides[2] = {q, k};
    const int n = k ? 2 : 1;
    for (int i = 0; i < n; ++i) {
        const rope_status_t st = check_side(sides[i], i ? "k" : "q", c);
        if (st != ROPE_OK) return st;
    }
    const bool rows = c.B > 0 && c.S > 0;
    const int e = size_of(c.dtype);
    const int64_t tokens[2] = {c.B, c.S};
    if (rows && L) {
        if (!c.cos || !c.sin || !c.cos_stride || !c.sin_stride)
            return fail(ROPE_ERR_NULLPTR, "cos, sin or their strides is null");
        if (span(tokens, c.cos_stride, 2, L, 0) < 0 || span(tokens, c.sin_stride, 2, L, 0) < 0)
            return fail(ROPE_ERR_INVALID, "strides of cos and sin must be >= 0 and in range");
        if (!aligned(c.cos, e) || !aligned(c.sin, e))
            return fail(ROPE_ERR_INVALID, "cos and sin must be aligned to their elements");
    }
    const bool wants = c.back && (q->weight_grad || (k && k->weight_grad));
    if (wants && !c.workspace) return fail(ROPE_ERR_NULLPTR, "workspace is null");
    if (!aligned(c.workspace, 16)) return fail(ROPE_ERR_INVALID, "workspace must be 16-byte aligned");
    if (!rows && !wants) return ROPE_OK;
    if (rows) {
        const rope_status_t st = check_overlap(sides, n, c);
        if (st != ROPE_OK) return st;
    }

    NormArgs a{};
    a.D = static_cast<int32_t>(c.D);
    a.n0 = static_cast<int32_t>(c.n0);
    a.n1 = static_cast<int32_t>(c.n1);
    a.start = static_cast<int32_t>(c.start);
    a.end = static_cast<int32_t>(c.end);
    a.weight32 = c.weight_dtype == ROPE_FP32;
    a.interleave = c.mode == ROPE_MODE_INTERLEAVE;
    a.eps = static_cast<float>(c.eps);
    a.inv_n = 1.0f / static_cast<float>(c.n1 - c.n0);
    a.sides = n;
    a.div_S = FastDiv::make(static_cast<uint32_t>(c.S > 0 ? c.S : 1));
    const int ve = 16 / e, half = static_cast<int>(L / 2);
    a.wide = c.D % ve == 0;
    bool wide_weight = true, wide_cs = false;
    for (int i = 0; i < n; ++i) {
        const rope_norm_rows_t* r = sides[i];
        const int64_t shape[3] = {c.B, c.S, r->heads};
        a.wide = a.wide && aligned(r->x, 16) && aligned(r->out, 16) && (!c.back || aligned(r->grad, 16));
        wide_weight = wide_weight && aligned(r->weight, 16);
        NormRows& s = a.side[i];
        for (int j = 0; j < 3; ++j) {
            s.x_st[j] = step(shape[j], r->x_stride[j]) * e;
            s.out_st[j] = step(shape[j], r->out_stride[j]) * e;
            s.grad_st[j] = c.back ? step(shape[j], r->grad_stride[j]) * e : 0;
            a.wide = a.wide && s.x_st[j] % 16 == 0 && s.out_st[j] % 16 == 0 && s.grad_st[j] % 16 == 0;
        }
        s.x = static_cast<const char*>(r->x);
        s.out = static_cast<char*>(r->out);
        s.grad = static_cast<const char*>(r->grad);
        s.weight = static_cast<const char*>(r->weight);
        s.rstd = r->rstd;
        s.heads = static_cast<int32_t>(r->heads);
    }
    if (L && rows) {
        a.cos = static_cast<const char*>(c.cos);
        a.sin = static_cast<const char*>(c.sin);
        wide_cs = aligned(c.cos, 16) && aligned(c.sin, 16);
        a.pairs_cs = aligned(c.cos, 2 * e) && aligned(c.sin, 2 * e);
        for (int j = 0; j < 2; ++j) {
            a.cos_st[j] = step(tokens[j], c.cos_stride[j]) * e;
            a.sin_st[j] = step(tokens[j], c.sin_stride[j]) * e;
            wide_cs = wide_cs && a.cos_st[j] % 16 == 0 && a.sin_st[j] % 16 == 0;
            a.pairs_cs = a.pairs_cs && a.cos_st[j] % (2 * e) == 0 && a.sin_st[j] % (2 * e) == 0;
        }
    }
    NormPlan p{};
    p.dtype = c.dtype;
    p.back = c.back;
    // The fast kernels where chunks are normed as a whole or not at all; pairs within a chunk (of
    // a slice of whole chunks, or pair by pair), or half-split pairs whose partners are whole
    // chunks, all normed or none.  Two prompts of 8192 tokens, 32 + 8 heads of 128 bf16,
    // 64 us so and 364 by the general kernels, which ask for each element; 16384 tokens' backward of
    // 16 + 4 heads 60 and 176.
    const bool whole = c.start % ve == 0 && wide_cs;
    const bool chunks_normed = a.wide && wide_weight && c.n0 % ve == 0 && c.n1 % ve == 0;
    const bool one_kind = (c.start >= c.n0 && c.end <= c.n1) || c.end <= c.n0 || c.start >= c.n1;
    p.turn = !chunks_normed                                            ? kTurnAny
             : L == 0 || (a.interleave && whole && L % ve == 0) ? kTurnNear
             : a.interleave && c.start % 2 == 0                        ? kTurnPairs
             : !a.interleave && whole && half % ve == 0 && one_kind    ? kTurnFar
                                                                       : kTurnAny;
    // The lanes of a row and their chunks: as few idle places as can be, then as few
    // chunks a lane as can be (more lanes at work for a row).
    const int chunks = static_cast<int>((c.D + ve - 1) / ve);
    const int few[] = {1, 2, 3, 4, 0}, many[] = {1, 2, 3, 5, 8, 0};
    int best = 1 << 30;
    for (const int* x = e == 4 ? many : few; *x; ++x)
        for (int log2 = 2; log2 <= 5; ++log2) {
            const int places = *x << log2;
            if (places >= chunks && places < best) best = places, p.chunks = *x, a.lanes_log2 = log2;
        }
    p.many = q->heads >= 2;
    const NormKernel kernel = norm_kernel(p);
    const char* err = nullptr;
    if (!kernel.f) return fail(ROPE_ERR_CUDA, "internal error: no kernel instance for this plan");
    for (int i = 0; i < n; ++i) {
        NormRows& s = a.side[i];
        s.groups = (s.heads + kernel.heads - 1) / kernel.heads;
        s.items = static_cast<uint32_t>(c.B * c.S * s.groups);
        s.div_groups = FastDiv::make(static_cast<uint32_t>(s.groups));
    }
    if (!c.back) {
        if (launch_norm_fwd(kernel, a, stream, &err) != ROPE_OK) return fail(ROPE_ERR_CUDA, "%s", err);
        return ROPE_OK;
    }
    int blocks = 0;
    NormJoin join{};
    join.lanes = a.n1 - a.n0;
    if (wants) {
        int sms = 0;
        if (norm_sm_count(&sms, &err) != ROPE_OK) return fail(ROPE_ERR_CUDA, "%s", err);
        int64_t need = 0;
        norm_workspace(c.n1 - c.n0, sms, &need);
        if (c.workspace_bytes < need)
            return fail(ROPE_ERR_INVALID, "workspace of %lld bytes; the call needs %lld",
                        (long long)c.workspace_bytes, (long long)need);
        float* part = static_cast<float*>(c.workspace);
        for (int i = 0; i < n; ++i)
            if (sides[i]->weight_grad) {
                a.side[i].part = part + int64_t(i) * sms * kNormBlocksPerSm * join.lanes;
                join.part[i] = a.side[i].part;
                join.out[i] = sides[i]->weight_grad;
            }
    }
    if (rows) {
        if (norm_blocks(kernel, a, &blocks, &err) != ROPE_OK ||
            launch_norm_bwd(kernel, a, blocks, stream, &err) != ROPE_OK)
            return fail(ROPE_ERR_CUDA, "%s", err);
    }
    join.blocks = blocks;
    if (wants && launch_norm_join(join, stream, &err) != ROPE_OK) return fail(ROPE_ERR_CUDA, "%s", err);
    return ROPE_OK;
}

}  // namespace
}  // namespace rope

extern "C" {

rope_status_t rope_partial_norm_fwd(const rope_norm_rows_t* q, const rope_norm_rows_t* k,
                                    rope_dtype_t dtype, rope_dtype_t weight_dtype, int64_t B,
                                    int64_t S, int64_t D, int64_t norm_start, int64_t norm_end,
                                    double eps, const void* cos, const void* sin,
                                    const int64_t cos_stride[2], const int64_t sin_stride[2],
                                    int64_t start, int64_t end, rope_mode_t mode,
                                    rope_stream_t stream) {
    return rope::norm(q, k, rope::Call{static_cast<int>(dtype), static_cast<int>(weight_dtype), B, S, D, norm_start,
                                       norm_end, eps, cos, sin, cos_stride, sin_stride, start, end,
                                       static_cast<int>(mode), false, nullptr, 0}, stream);
}

rope_status_t rope_partial_norm_bwd(const rope_norm_rows_t* q, const rope_norm_rows_t* k,
                                    rope_dtype_t dtype, rope_dtype_t weight_dtype, int64_t B,
                                    int64_t S, int64_t D, int64_t norm_start, int64_t norm_end,
                                    const void* cos, const void* sin, const int64_t cos_stride[2],
                                    const int64_t sin_stride[2], int64_t start, int64_t end,
                                    rope_mode_t mode, void* workspace, int64_t workspace_bytes,
                                    rope_stream_t stream) {
    return rope::norm(q, k, rope::Call{static_cast<int>(dtype), static_cast<int>(weight_dtype), B, S, D, norm_start,
                                       norm_end, 0.0, cos, sin, cos_stride, sin_stride, start, end,
                                       static_cast<int>(mode), true, workspace, workspace_bytes}, stream);
}

rope_status_t rope_partial_norm_workspace(int64_t normed, int32_t sm_count, int64_t* bytes) {
    using namespace rope;
    clear_error();
    if (!bytes) return fail(ROPE_ERR_NULLPTR, "bytes is null");
    if (normed < 1 || normed > 1024) return fail(ROPE_ERR_INVALID, "normed=%lld must be 1 .. 1024", (long long)normed);
    if (sm_count < 0) return fail(ROPE_ERR_INVALID, "sm_count is negative");
    int sms = sm_count;
    const char* err = nullptr;
    if (sms == 0 && norm_sm_count(&sms, &err) != ROPE_OK) return fail(ROPE_ERR_CUDA, "%s", err);
    return norm_workspace(normed, sms, bytes);
}

}  // extern "C"
