/*
 * rope_step.h -- C ABI of the operators on either side of the paged cache of
 * rope_serving.h in a model's step:
 *
 *   rope_partial_norm_fwd / _bwd      root-mean-square norm of query and key rows and
 *                                     the rotation of a slice of them, in one pass
 *   rope_partial_cache_grow / _trim   pages, slots and positions for a batch's new
 *                                     tokens, made on the device, and pages given back
 *   rope_partial_latent_attention     attention over a cache of latent rows, one for
 *                                     all heads, whose first lanes are the values
 *
 * Conventions are those of rope_partial.h and rope_serving.h: plain C, device
 * pointers on the current CUDA device, int64 sizes, ELEMENT strides, the
 * caller's stream, nothing allocated, nothing synchronised; arguments are
 * checked on the host before anything is launched, an invalid call changes
 * nothing and returns an error status, and rope_last_error_message()
 * describes it.
 */
#ifndef ROPE_STEP_H
#define ROPE_STEP_H

#include "rope_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Norm and rotation of rows in one pass
 * ------------------------------------------------------------------------ */

/* The rows of the queries or of the keys: (B, S, heads, D) with ELEMENT strides
   of the first three dims (>= 0; that of a dim of one is not looked at) and a
   contiguous last dim. */
typedef struct {
    const void* x;          /* the rows before the norm */
    void* out;              /* forward: the result; backward: the gradient of x */
    const void* grad;       /* backward: the gradient of the result; else not used */
    const void* weight;     /* one factor for each normed lane, or null (all 1) */
    float* rstd;            /* (B, S, heads) contiguous, 1 / root mean square of each row:
                               forward: written, unless null; backward: read */
    float* weight_grad;     /* backward: the gradient of the weight (one fp32 for each
                               normed lane), overwritten; null: not wanted */
    int64_t heads;
    int64_t x_stride[3], out_stride[3], grad_stride[3];
} rope_norm_rows_t;

/*
 * rope_partial_norm_fwd -- for each row x of the queries and, where k is not
 * null, of the keys:
 *
 *     r   = 1 / sqrt(eps + sum of x_j^2 over the normed lanes / their number)
 *     y_j = x_j r weight_j on the lanes [norm_start, norm_end), x_j elsewhere
 *     out = y with the lanes [start, end) rotated as in rope_partial_inplace_fwd_mode
 *
 * Everything is computed in fp32 and rounded once when it is stored (rows whose
 * squares fp32 does not hold are not normed rightly).
 *
 *   q, k           k may be null.  Both have D lanes, and the same norm and slice.
 *   dtype          of x, out, grad, cos and sin: bf16, fp16 or fp32
 *   weight_dtype   of the weights: dtype, or fp32
 *   D              1 .. 1024, odd ones too
 *   norm_start, norm_end   0 <= norm_start < norm_end <= D
 *   eps            >= 0 and finite
 *   cos, sin       rows of end - start elements of `dtype` at ELEMENT strides
 *                  {batch, token} (>= 0; 0: one row for all); null when start == end
 *   start, end, mode   as for rope_partial_inplace_fwd_mode; any start
 *
 * out may be x itself (the same address and strides: in place); otherwise no
 * output may share a byte with another output or with anything that is read.
 * Rows of 16-byte aligned addresses, strides and lengths are the fast case.  A
 * batch without rows is a no-op.
 */
rope_status_t rope_partial_norm_fwd(const rope_norm_rows_t* q, const rope_norm_rows_t* k,
                                    rope_dtype_t dtype, rope_dtype_t weight_dtype, int64_t B,
                                    int64_t S, int64_t D, int64_t norm_start, int64_t norm_end,
                                    double eps, const void* cos, const void* sin,
                                    const int64_t cos_stride[2], const int64_t sin_stride[2],
                                    int64_t start, int64_t end, rope_mode_t mode,
                                    rope_stream_t stream);

/*
 * rope_partial_norm_bwd -- the gradients of the forward.  With g the transposed
 * rotation of grad (the forward's cos and sin), u_j = x_j rstd and n normed
 * lanes:
 *
 *     weight_grad_j = sum over all rows of g_j u_j
 *     out_j = rstd (weight_j g_j - u_j sum_i(weight_i g_i u_i) / n) on the normed
 *     lanes, g_j elsewhere
 *
 * x, rstd and grad are read, out is written; out may be grad itself (the same
 * address and strides).  cos and sin get no gradient.  Sums are fp32, in an
 * order that depends on sizes and the device alone, so a call repeated gives
 * the same bits.
 *
 *   workspace   rope_partial_norm_workspace() bytes, 16-byte aligned, for this
 *               call alone until it has run; its contents do not matter.  Null
 *               when no weight_grad is wanted.
 * A batch without rows gives weight gradients of zero.
 */
rope_status_t rope_partial_norm_bwd(const rope_norm_rows_t* q, const rope_norm_rows_t* k,
                                    rope_dtype_t dtype, rope_dtype_t weight_dtype, int64_t B,
                                    int64_t S, int64_t D, int64_t norm_start, int64_t norm_end,
                                    const void* cos, const void* sin, const int64_t cos_stride[2],
                                    const int64_t sin_stride[2], int64_t start, int64_t end,
                                    rope_mode_t mode, void* workspace, int64_t workspace_bytes,
                                    rope_stream_t stream);

/* The bytes of workspace that a backward with `normed` = norm_end - norm_start lanes
   needs on the current device (sm_count > 0: on a device with that many SMs, without
   touching the GPU). */
rope_status_t rope_partial_norm_workspace(int64_t normed, int32_t sm_count, int64_t* bytes);

/* ------------------------------------------------------------------------
 * Pages of the cache, slots and positions for a batch of requests
 * ------------------------------------------------------------------------ */

/*
 * rope_partial_cache_grow -- for R requests that hold kv_len[r] cached rows and get
 * n[r] new tokens each: pages for them, and what the calls of rope_serving.h want to
 * know of the batch.  A request of `len` rows holds ceil(len / page_size) pages,
 * the first entries of its row of the page table.  It needs
 *
 *     need[r] = ceil((kv_len[r] + n[r]) / page_size) - ceil(kv_len[r] / page_size)
 *
 * more.  Pages come from the top of the stack free_pages[0 .. *free_count), in the
 * order of the requests: need[r] of them are granted when need[r] is 0, or when
 * they and those that all earlier requests need (granted or not) are there.  A request
 * whose pages would pass max_pages is not granted and takes part in nothing.  So a
 * batch that asks for too much serves a front part of its requests, and those that need
 * no page.
 *
 *   kv_len      device pointer to R int32, in place: granted requests grow by n[r].
 *               Lengths are taken as within [0, max_pages * page_size].
 *   n           device pointer to R int32; a negative number counts as 0
 *   page_table  (R, max_pages) int32, rows page_table_stride apart, in place: the new
 *               pages of granted requests are written behind their old ones
 *   free_pages  device pointer to free_capacity int32 page numbers; free_count to
 *               one int32, in place, which is taken as within [0, free_capacity]
 *   q_start     R + 1 int32, written: offsets of the requests' tokens, those of
 *               requests that are not granted included (q_start[R]: how many there are;
 *               sums that pass 2^31 - 1 stay there)
 *   slots       T int64, written: the slot (page * page_size + place) of every token of
 *               a granted request; -1, which the cache calls skip, for the
 *               tokens of others and for places from q_start[R] on.  Tokens from T on
 *               are left out.
 *   positions   T int32, or null, written: kv_len[r] (before) + i for token i of
 *               request r, granted or not; 0 from q_start[R] on
 *   granted     R int32, or null, written: 1 or 0
 *
 * Everything is read and written on the device, nothing on the host: a call captured in
 * a graph may be replayed for other batches of R requests.  Sizes: page_size >= 1,
 * max_pages * page_size < 2^31, R < 2^24, T < 2^31.  Nothing of what is written may
 * share a byte with anything else.  R == 0 writes q_start[0] = 0 and the places of slots
 * and positions.
 */
rope_status_t rope_partial_cache_grow(int32_t* kv_len, const int32_t* n, int64_t R,
                                      int32_t* page_table, int64_t max_pages,
                                      int64_t page_table_stride, const int32_t* free_pages,
                                      int64_t free_capacity, int32_t* free_count, int64_t page_size,
                                      int32_t* q_start, int64_t* slots, int32_t* positions,
                                      int64_t T, int32_t* granted, rope_stream_t stream);

/*
 * rope_partial_cache_trim -- requests that keep new_len[r] of their rows (drafted
 * tokens that were not accepted; 0: a request that has ended) give back the pages
 * behind them:
 *
 *     keep[r] = min(max(new_len[r], 0), kv_len[r])
 *
 * The entries [ceil(keep / page_size), ceil(kv_len / page_size)) of a request's row go
 * onto the stack and become -1 in the table, and kv_len[r] becomes keep[r].  The pages
 * lie on the stack so that a call of rope_partial_cache_grow that is taken back
 * leaves the stack as it was: those of the first request uppermost, and of a
 * request's the earliest.  Pages that would pass free_capacity, which no page that came
 * from the stack does, are dropped.
 *
 * Arguments as above; new_len is a device pointer to R int32 (not kv_len itself, which
 * is written).  Entries are not looked into: what the table holds goes onto the stack.
 * R == 0 is a no-op.
 */
rope_status_t rope_partial_cache_trim(int32_t* kv_len, const int32_t* new_len, int64_t R,
                                      int32_t* page_table, int64_t max_pages,
                                      int64_t page_table_stride, int32_t* free_pages,
                                      int64_t free_capacity, int32_t* free_count, int64_t page_size,
                                      rope_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention over latent rows
 * ------------------------------------------------------------------------ */

/*
 * rope_partial_latent_attention -- rope_partial_tree_attention over a cache that has one
 * row a token for all query heads, of which the first v_dim lanes are the value:
 *
 *     s_j = scale * q . k_j        out = sum_j exp(s_j) k_j[0 .. v_dim) / sum_j exp(s_j)
 *
 * (keys and values of all heads made from one latent vector, with the heads' own
 * matrices multiplied into q and out; the row's other lanes, a rotated part that
 * all heads share, say, count for the score alone).
 *
 *   cache        one head, no values (v null, v_dim 0); any of its types.  Such rows
 *                are written by rope_partial_cache_write and read by
 *                rope_partial_cache_read as any keys are.
 *   v_dim        the lanes of the value, and of a row of out
 *   scale        the model's own: with matrices multiplied into q, that of the heads' query
 *                rows before the product (1 / sqrt(192) for heads of 128 + 64 lanes), not of k_dim
 *   other arguments, requests, trees, lengths, masks and the workspace
 *                as for rope_partial_tree_attention: chains without a tree, tokens that
 *                see no row (0 and -inf), tokens outside every request (left as
 *                they are), captured calls, and that a row has no effect on a token that
 *                does not see it.  max_q is a hint; sums are fp32; waits are
 *                bounded.
 *
 * Types: a 16-bit cache must have the type of q; an 8-bit cache (whose scales may have any
 * sign) goes with either.  Sizes: k_dim and v_dim multiples of 16, 16 <= v_dim <= k_dim <=
 * 576, v_dim <= 512.  Rows of q, out and the cache must start on 16-byte boundaries.
 * Products run on tensor cores in bf16 (bf16 caches) or fp16 (the others) with fp32
 * accumulation.  exp(s), for 8-bit caches times the row's scale, is rounded to that type
 * once; in fp16 what is below 2^-21 of the token's largest loses bits and below 2^-31
 * vanishes (scales below 2^-80 are as small there as they are).  For 8-bit caches q is
 * rounded to fp16 after a power of two that brings the row's largest lane to [1, 2).
 * 16-bit rows of a multiple of 64 lanes in pages of a multiple of 8 rows are the fast case
 * (the larger the power of two that divides the page, to 64, the larger the copies).
 */
rope_status_t rope_partial_latent_attention(const rope_kv_cache_t* cache, const void* q,
                                            rope_dtype_t dtype, int64_t Tq, int64_t Hq, int64_t v_dim,
                                            const int64_t q_stride[2], const int32_t* q_start,
                                            const int32_t* kv_len, int64_t R, int64_t max_q,
                                            const int32_t* page_table, int64_t max_pages,
                                            int64_t page_table_stride, const int64_t* tree,
                                            int64_t tree_words, void* out,
                                            const int64_t out_stride[2], float* lse, double scale,
                                            void* workspace, int64_t workspace_bytes,
                                            rope_stream_t stream);

/* The bytes of workspace that such a call needs on the current device (sm_count > 0: on a
   device with that many SMs, without touching the GPU). */
rope_status_t rope_partial_latent_attention_workspace(const rope_kv_cache_t* cache,
                                                      rope_dtype_t dtype, int64_t Hq, int64_t v_dim,
                                                      int64_t max_q, int32_t sm_count,
                                                      int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_STEP_H */
