// rope_latent_host.cpp -- the C ABI entry points of include/rope_step.h for the attention
// over latent rows: argument checks, the choice of kernel and the launches.  No CUDA call
// is made for a rejected or empty call.
#include <float.h>
#include <math.h>

#include "rope_check.h"
#include "rope_latent.h"

namespace rope {
namespace {

constexpr int64_t kInt = (int64_t(1) << 31) - 1;

rope_status_t latent_plan(const rope_kv_cache_t* c, int dtype, int64_t Hq, int64_t v_dim, int64_t max_q,
                          LatentPlan* p) {
    if (dtype != ROPE_BF16 && dtype != ROPE_FP16)
        return fail(ROPE_ERR_INVALID, "attention takes bf16 (0) or fp16 (1), not dtype %d", dtype);
    if (code_size(c->dtype) == 2 && c->dtype != dtype)
        return fail(ROPE_ERR_INVALID, "a 16-bit cache must have the type of q (cache %d, q %d)", int(c->dtype), dtype);
    if (c->heads != 1 || c->v_dim != 0)
        return fail(ROPE_ERR_INVALID, "a cache of latent rows has one head and no values of its own (heads=%lld "
                    "v_dim=%lld)", (long long)c->heads, (long long)c->v_dim);
    if (c->k_dim > kLatentLanes || v_dim > kLatentValues || v_dim > c->k_dim || v_dim < 16 || c->k_dim % 16 ||
        v_dim % 16)
        return fail(ROPE_ERR_INVALID, "k_dim=%lld and v_dim=%lld must be multiples of 16 with 16 <= v_dim <= k_dim <= "
                    "%d and v_dim <= %d", (long long)c->k_dim, (long long)v_dim, kLatentLanes, kLatentValues);
    if (Hq < 1 || Hq > (1 << 20)) return fail(ROPE_ERR_INVALID, "Hq=%lld must be positive", (long long)Hq);
    if (max_q < 1 || max_q > kInt) return fail(ROPE_ERR_INVALID, "max_q=%lld must be positive", (long long)max_q);
    *p = choose_latent(c->dtype, max_q * Hq, c->k_dim, c->pages, c->page_size);
    return ROPE_OK;
}

rope_status_t latent_attention(const rope_kv_cache_t* c, const void* q, int dtype, int64_t Tq, int64_t Hq,
                               int64_t v_dim, const int64_t* q_stride, const int32_t* q_start, const int32_t* kv_len,
                               int64_t R, int64_t max_q, const int32_t* page_table, int64_t max_pages,
                               int64_t table_stride, const int64_t* tree, int64_t words, void* out,
                               const int64_t* out_stride, float* lse, double scale, void* workspace,
                               int64_t workspace_bytes, rope_stream_t stream) {
    clear_error();
    int64_t kb, vb;
    rope_status_t st = check_cache(c, &kb, &vb);
    if (st != ROPE_OK) return st;
    LatentPlan p{};
    st = latent_plan(c, dtype, Hq, v_dim, max_q, &p);
    if (st != ROPE_OK) return st;
    if (Tq < 0 || Tq > (kInt - 64) / Hq || R < 0 || R > (1 << 24))
        return fail(ROPE_ERR_INVALID, "Tq=%lld query tokens, R=%lld requests", (long long)Tq, (long long)R);
    if (max_pages < 0 || max_pages > kInt || max_pages * c->page_size > kInt - 1024)
        return fail(ROPE_ERR_INVALID, "%lld pages of %lld tokens a request exceed 2^31 rows", (long long)max_pages,
                    (long long)c->page_size);
    if (c->pages > kInt) return fail(ROPE_ERR_INVALID, "more than 2^31 pages");
    if (table_stride < 0 || (R > 1 && table_stride < max_pages) || table_stride > kMaxSize)
        return fail(ROPE_ERR_INVALID, "page_table_stride %lld is less than max_pages %lld", (long long)table_stride,
                    (long long)max_pages);
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
    const int64_t so = span(shape, out_stride, 2, v_dim, v_dim);
    if (sq < 0 || so < 0)
        return fail(ROPE_ERR_INVALID, "strides of q and out must be >= 0, and keep the rows of out apart");
    bool ok = aligned(q, 16) && aligned(out, 16) && aligned(c->k, 16) && aligned(workspace, 16);
    const int64_t slots[3] = {c->pages, c->page_size, 1};
    for (int i = 0; i < 2; ++i)
        ok = ok && step(shape[i], q_stride[i]) * 2 % 16 == 0 && step(shape[i], out_stride[i]) * 2 % 16 == 0 &&
             step(slots[i], c->k_stride[i]) * ce % 16 == 0;
    if (!ok)
        return fail(ROPE_ERR_INVALID, "the rows of q, out and the cache and the workspace must start on 16-byte "
                    "boundaries");
    if (!aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4) || !aligned(tree, 8) || !aligned(lse, 4))
        return fail(ROPE_ERR_INVALID, "q_start, kv_len, page_table, tree and lse must be aligned to their elements");
    // out, lse and the workspace are written while everything else is read
    const struct { const void* p; int64_t n; } wr[3] = {
        {out, so * 2}, {lse, lse ? Tq * Hq * 4 : 0}, {workspace, workspace_bytes}};
    const struct { const void* p; int64_t n; } rd[4] = {
        {q_start, (R + 1) * 4}, {kv_len, R * 4},
        {page_table, max_pages ? ((R - 1) * table_stride + max_pages) * 4 : 0},
        {tree, tree ? Tq * words * 8 : 0}};
    const Rows qr = rows_of(q, Tq, Hq, q_stride, c->k_dim, 2), outr = rows_of(out, Tq, Hq, out_stride, v_dim, 2);
    bool hit = rows_overlap(qr, outr) || overlaps(q, sq * 2, wr[1].p, wr[1].n) || overlaps(q, sq * 2, wr[2].p, wr[2].n);
    for (int i = 0; i < 3; ++i) {
        hit = hit || in_cache(c, kb, vb, wr[i].p, wr[i].n);
        for (const auto& r : rd) hit = hit || overlaps(wr[i].p, wr[i].n, r.p, r.n);
        for (int j = 0; j < i; ++j) hit = hit || overlaps(wr[i].p, wr[i].n, wr[j].p, wr[j].n);
    }
    if (hit)
        return fail(ROPE_ERR_INVALID, "out, lse and workspace must not overlap each other or anything that is read");

    const char* err = nullptr;
    int blocks = 0;
    if (latent_blocks(p, 0, &blocks, &err) != ROPE_OK) return fail(ROPE_ERR_CUDA, "%s", err);
    const int64_t need = latent_workspace(p, blocks);
    if (workspace_bytes < need)
        return fail(ROPE_ERR_INVALID, "workspace of %lld bytes; the call needs %lld", (long long)workspace_bytes,
                    (long long)need);

    TreeArgs a{};
    // (no pages: no row is read, but the kernel forms an address all the same)
    a.k = a.v = static_cast<const char*>(c->pages ? c->k : q);
    a.ks = a.vs = c->pages ? c->k_scale : static_cast<const float*>(q);
    for (int i = 0; i < 3; ++i) {
        a.k_st[i] = a.v_st[i] = step(slots[i], c->k_stride[i]) * ce;
        a.ks_st[i] = a.vs_st[i] = step(slots[i], c->k_scale_stride[i]);
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
    a.Hk = 1;
    a.G = a.Hq = static_cast<int32_t>(Hq);
    a.Dk = static_cast<int32_t>(c->k_dim);
    a.Dv = static_cast<int32_t>(v_dim);
    a.pages = static_cast<int32_t>(c->pages);
    a.page_size = static_cast<int32_t>(c->page_size);
    a.max_len = static_cast<int32_t>(max_pages * c->page_size);
    a.div_page = FastDiv::make(static_cast<uint32_t>(c->page_size));
    a.div_group = FastDiv::make(static_cast<uint32_t>(Hq));
    a.scale_log2 = scale_log2;
    a.bf16 = dtype == ROPE_BF16;
    if (launch_latent(p, a, workspace, blocks, stream, &err) != ROPE_OK) return fail(ROPE_ERR_CUDA, "%s", err);
    return ROPE_OK;
}

}  // namespace
}  // namespace rope

extern "C" {

rope_status_t rope_partial_latent_attention(const rope_kv_cache_t* cache, const void* q,
                                            rope_dtype_t dtype, int64_t Tq, int64_t Hq, int64_t v_dim,
                                            const int64_t q_stride[2], const int32_t* q_start,
                                            const int32_t* kv_len, int64_t R, int64_t max_q,
                                            const int32_t* page_table, int64_t max_pages,
                                            int64_t page_table_stride, const int64_t* tree,
                                            int64_t tree_words, void* out,
                                            const int64_t out_stride[2], float* lse, double scale,
                                            void* workspace, int64_t workspace_bytes,
                                            rope_stream_t stream) {
    return rope::latent_attention(cache, q, static_cast<int>(dtype), Tq, Hq, v_dim, q_stride, q_start, kv_len, R,
                                  max_q, page_table, max_pages, page_table_stride, tree, tree_words, out, out_stride,
                                  lse, scale, workspace, workspace_bytes, stream);
}

rope_status_t rope_partial_latent_attention_workspace(const rope_kv_cache_t* cache,
                                                      rope_dtype_t dtype, int64_t Hq, int64_t v_dim,
                                                      int64_t max_q, int32_t sm_count,
                                                      int64_t* bytes) {
    using namespace rope;
    clear_error();
    if (!bytes) return fail(ROPE_ERR_NULLPTR, "bytes is null");
    if (sm_count < 0) return fail(ROPE_ERR_INVALID, "sm_count is negative");
    int64_t kb, vb;
    rope_status_t st = check_cache(cache, &kb, &vb);
    if (st != ROPE_OK) return st;
    LatentPlan p{};
    st = latent_plan(cache, static_cast<int>(dtype), Hq, v_dim, max_q, &p);
    if (st != ROPE_OK) return st;
    const char* err = nullptr;
    int blocks = 0;
    if (latent_blocks(p, sm_count, &blocks, &err) != ROPE_OK) return fail(ROPE_ERR_CUDA, "%s", err);
    *bytes = latent_workspace(p, blocks);
    return ROPE_OK;
}

}  // extern "C"
