/*
 * rope_serving.h -- C ABI of the operators around the in-place partial rotary
 * embedding that a model with several position axes, or a decoding step over
 * a paged cache, runs next to it:
 *
 *   rope_partial_inplace_{fwd,bwd}_axes   rotary positions with several axes
 *   rope_partial_cache_write / _read      a paged cache of rotated keys and of
 *                                         values, 16-bit or quantised to 8 bits
 *   rope_partial_tree_attention           attention of drafted tokens (a tree,
 *                                         a chain or single tokens) over it
 *   rope_partial_tree_mask                a tree's ancestor bits, on the host
 *
 * Conventions are those of rope_partial.h: plain C, device pointers on the
 * current CUDA device, int64 sizes, ELEMENT strides, the caller's stream,
 * nothing allocated, nothing synchronised; arguments are checked on the host
 * before anything is launched, an invalid call changes nothing and returns an
 * error status, and rope_last_error_message() describes it.  Values that only
 * the device can see (slots, page numbers, lengths) are checked by the
 * kernels against the sizes given here, so that no value of theirs reads or
 * writes outside the tensors.
 */
#ifndef ROPE_SERVING_H
#define ROPE_SERVING_H

#include "rope_partial.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Rotary positions with several axes (time, height and width of a video;
 * height and width of an image; text beside them)
 * ------------------------------------------------------------------------ */

/* Which pairs of the slice belong to which axis.  Blocked: the first
   sections[0] pairs to axis 0, the next sections[1] to axis 1, and so on.
   Interleaved: pairs are dealt to the axes in turn, an axis dropping out once
   it has its sections[a] pairs. */
typedef enum {
    ROPE_AXES_BLOCKED = 0,
    ROPE_AXES_INTERLEAVED = 1
} rope_axes_order_t;

/* The frequency of a pair.  Shared: omega = base^(-2k/L) with k the pair's
   index in the slice, one spectrum that the axes share out.  Own:
   omega = base^(-j/sections[a]) for the j-th pair of axis a, so that every
   axis has a whole spectrum. */
typedef enum {
    ROPE_SPECTRUM_SHARED = 0,
    ROPE_SPECTRUM_OWN = 1
} rope_spectrum_t;

#define ROPE_MAX_AXES 4

/*
 * rope_partial_inplace_fwd_axes / _bwd_axes -- rope_partial_inplace_fwd_pos
 * / _bwd_pos with one position per axis: pair k of the slice, which belongs
 * to axis a, turns by theta = positions[a][b][s] * omega.  Both lanes of a
 * pair use cos(theta) and sin(theta); the backward is the transposed
 * rotation.
 *
 *   axes        1 .. ROPE_MAX_AXES
 *   sections    host array of `axes` pair counts, each >= 0, that add up to
 *               L / 2 (L = end - start)
 *   positions   device pointer to int32, shape pos_shape = {axes, B or 1,
 *               S or 1} with ELEMENT strides pos_stride (>= 0; that of a
 *               broadcast dim is ignored)
 *   other       as for rope_partial_inplace_fwd_pos: in place, x contiguous
 *               (B, S, N, D), any start, both rotary modes, base > 0, the
 *               error bound on cos and sin for |position| < 2^24, the
 *               empty-call rule, status codes.  x and the positions must not
 *               share a byte.
 *
 * With one axis and sections = {L / 2} the results are those of the
 * positions call.
 */
rope_status_t rope_partial_inplace_fwd_axes(void* x, const int32_t* positions, rope_dtype_t dtype,
                                            int64_t B, int64_t S, int64_t N, int64_t D,
                                            int32_t axes, const int32_t* sections,
                                            const int64_t pos_shape[3], const int64_t pos_stride[3],
                                            rope_axes_order_t order, rope_spectrum_t spectrum,
                                            double base, int64_t start, int64_t end,
                                            rope_mode_t mode, rope_stream_t stream);

rope_status_t rope_partial_inplace_bwd_axes(void* grad, const int32_t* positions,
                                            rope_dtype_t dtype, int64_t B, int64_t S, int64_t N,
                                            int64_t D, int32_t axes, const int32_t* sections,
                                            const int64_t pos_shape[3], const int64_t pos_stride[3],
                                            rope_axes_order_t order, rope_spectrum_t spectrum,
                                            double base, int64_t start, int64_t end,
                                            rope_mode_t mode, rope_stream_t stream);

/* ------------------------------------------------------------------------
 * The paged cache
 * ------------------------------------------------------------------------ */

/* Storage types of a cache.  The 16-bit types hold the values themselves;
   the 8-bit types hold a row's values divided by one fp32 scale per (token,
   head): FP8 is e4m3 (largest value 448), INT8 uses -127 .. 127. */
typedef enum {
    ROPE_CACHE_BF16 = 0,
    ROPE_CACHE_FP16 = 1,
    ROPE_CACHE_FP8 = 3,
    ROPE_CACHE_INT8 = 4
} rope_cache_dtype_t;

/* A cache of `pages` pages of `page_size` token slots, with `heads` key and
   value rows per slot: k is (pages, page_size, heads, k_dim), v is (pages,
   page_size, heads, v_dim), in ELEMENT strides for the first three dims and
   a contiguous last dim, so that a head-major page is a matter of strides.
   k_scale and v_scale, (pages, page_size, heads), are needed for the 8-bit
   types (values' scales are not negative) and null for the others.  A cache without values has v == null and
   v_dim == 0.  Slot s is token s % page_size of page s / page_size. */
typedef struct {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t pages, page_size, heads, k_dim, v_dim;
    int64_t k_stride[3], v_stride[3];
    int64_t k_scale_stride[3], v_scale_stride[3];
    int32_t dtype; /* rope_cache_dtype_t */
    int32_t reserved; /* 0 */
} rope_kv_cache_t;

/*
 * rope_partial_cache_write -- rotate lanes [start, end) of T new keys and
 * put them and their values into the cache.
 *
 *   k, v       device pointers to (T, heads, k_dim) and (T, heads, v_dim) of
 *              `dtype` (bf16, fp16 or fp32), ELEMENT strides k_stride and
 *              v_stride of the first two dims, contiguous last dim; read
 *              only, unlike the in-place calls.  v is null iff v_dim == 0.
 *   slots      device pointer to T int64 slots.  A slot outside
 *              [0, pages * page_size) (-1 for padding, say) skips its token.
 *              The other slots must differ from each other.
 *   cos, sin   device pointers to rows of L = end - start elements of
 *              `dtype`, cos_stride / sin_stride ELEMENTS apart per token (0:
 *              one row for all); null when start == end (no rotation).
 *              Rounding is that of rope_partial_inplace_fwd, except that the
 *              result stays in fp32 until it is stored.
 *   start, end, mode   as for rope_partial_inplace_fwd_mode, on k_dim lanes.
 *
 * Stored values: a 16-bit cache rounds each fp32 value once.  An 8-bit cache
 * takes m = max(largest |value| of the row, 2^-100), stores the fp32 scale
 * m / top (top = 448 or 127) and each value times the fp32 number top / m,
 * rounded to the nearest even code within [-top, top].  A row with an
 * infinity or a NaN stores a NaN scale and codes of 0, so that it reads back
 * as NaN.
 *
 * Sizes: k_dim and v_dim <= 1024, odd ones too.
 * The inputs must not overlap the cache.  T == 0 is a no-op.
 */
rope_status_t rope_partial_cache_write(const rope_kv_cache_t* cache, const void* k, const void* v,
                                       rope_dtype_t dtype, int64_t T, const int64_t k_stride[2],
                                       const int64_t v_stride[2], const int64_t* slots,
                                       const void* cos, const void* sin, int64_t cos_stride,
                                       int64_t sin_stride, int64_t start, int64_t end,
                                       rope_mode_t mode, rope_stream_t stream);

/*
 * rope_partial_cache_read -- the rows at T slots as numbers: each code times
 * its row's scale (a 16-bit cache: the value), rounded once to `dtype`, into
 * k (T, heads, k_dim) and v (T, heads, v_dim), ELEMENT strides as above.  A
 * null k or v leaves that half out.  A slot outside the cache gives a row of
 * zeros.  The outputs must not overlap each other, the cache or the slots;
 * their token and head strides must keep rows apart.
 */
rope_status_t rope_partial_cache_read(const rope_kv_cache_t* cache, const int64_t* slots, int64_t T,
                                      void* k, void* v, rope_dtype_t dtype,
                                      const int64_t k_stride[2], const int64_t v_stride[2],
                                      rope_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention of drafted tokens over the cache
 * ------------------------------------------------------------------------ */

/*
 * rope_partial_tree_attention -- for each of R requests, attention of its
 * drafted tokens over its cached rows.  Request r has the query tokens
 * [q_start[r], q_start[r+1]) (n of them, any number from 0) and kv_len[r]
 * cached rows, of which the last n are the drafted tokens' own (written
 * before this call); row j lies at slot j % page_size of page
 * page_table[r][j / page_size].  Drafted token i sees row j when
 * j < kv_len[r] - n (the context), or, with jj = j - (kv_len[r] - n), when
 * bit jj of its tree words is set (bit jj % 64 of word jj / 64; a row past
 * the last word is not seen), or, without a tree, when jj <= i: a chain,
 * which is ordinary causal decoding.  Then, for query head h and key head
 * h / (Hq / heads):
 *
 *     s_j = scale * q . k_j        out = sum_j exp(s_j) v_j / sum_j exp(s_j)
 *     lse = log(sum_j exp(s_j))    over the rows j that the token sees
 *
 * A token that sees no row gets out = 0 and lse = -inf.  A row that a token
 * does not see has no effect on it, whatever the row holds.
 *
 *   q            (Tq, Hq, k_dim) of `dtype` (bf16 or fp16), ELEMENT strides
 *                q_stride of the first two dims, contiguous last dim
 *   q_start      R + 1 int32 offsets that do not decrease; kv_len: R int32;
 *                both on the device.  Lengths are clamped to the page table
 *                (max_pages * page_size rows), offsets to [0, Tq].
 *   max_q        the most drafted tokens that a request has (a hint, > 0:
 *                it chooses the kernel; a wrong one costs time only)
 *   page_table   (R, max_pages) int32, rows page_table_stride apart.  A page
 *                number outside the cache counts as rows of zeros.
 *   tree         (Tq, tree_words) int64 bits, contiguous, or null for a chain
 *   out          (Tq, Hq, v_dim) of `dtype`, strides out_stride; tokens
 *                outside every request are left as they are
 *   lse          (Tq, Hq) fp32, contiguous, or null
 *   scale        > 0; times log2(e) a normal fp32 number
 *   workspace    at least rope_partial_tree_attention_workspace() bytes,
 *                16-byte aligned, for this call alone until it has run; its
 *                contents do not matter
 *
 * Types: a 16-bit cache must have the type of q; an 8-bit cache goes with
 * either.  Sizes: k_dim and v_dim multiples of 16, v_dim <= k_dim <= 256;
 * heads divides Hq.  Rows of q, out and the cache must start on 16-byte
 * boundaries.  Sums are fp32; the products of q with k and of exp(s) with v
 * run on tensor cores in bf16 (bf16 caches) or fp16 (the others) with fp32
 * accumulation, exp(s) being rounded to that type once.  In fp16, what is
 * rounded (for 8-bit caches exp(s) times the value's scale) is counted from the
 * token's largest: below 2^-29 (2^-21 for more than 16 query rows a key head) of it
 * the rounding grows, below 2^-39 (2^-31) the row vanishes.  For 8-bit
 * caches q is rounded to fp16 after a power of two that brings the row's
 * largest lane to [1, 2).  Pages of a multiple
 * of 8 rows, and up to 192 + 128 lanes, are the fast case: others read the
 * cache once for each 16 query rows of a key head.  A call captured in a graph
 * may be replayed with other contents of the device arrays.  Waits inside the
 * kernels are bounded: should nothing move for seconds (the device is at fault), the
 * results that depend on it are NaN, and the call ends.
 */
rope_status_t rope_partial_tree_attention(const rope_kv_cache_t* cache, const void* q,
                                          rope_dtype_t dtype, int64_t Tq, int64_t Hq,
                                          const int64_t q_stride[2], const int32_t* q_start,
                                          const int32_t* kv_len, int64_t R, int64_t max_q,
                                          const int32_t* page_table, int64_t max_pages,
                                          int64_t page_table_stride, const int64_t* tree,
                                          int64_t tree_words, void* out,
                                          const int64_t out_stride[2], float* lse, double scale,
                                          void* workspace, int64_t workspace_bytes,
                                          rope_stream_t stream);

/* The bytes of workspace that a call with this cache, `dtype`, Hq and max_q
   needs on the current device (sm_count > 0: on a device with that many SMs,
   without touching the GPU).  It does not depend on lengths. */
rope_status_t rope_partial_tree_attention_workspace(const rope_kv_cache_t* cache,
                                                    rope_dtype_t dtype, int64_t Hq, int64_t max_q,
                                                    int32_t sm_count, int64_t* bytes);

/* The tree words of one request from its parents: parents[i] in [-1, i) is
   the drafted token that token i follows (-1: the context).  words[i *
   tree_words + w] gets the bits of i and of all its ancestors.  tree_words
   >= ceil(n / 64).  Host only: no CUDA call. */
rope_status_t rope_partial_tree_mask(const int32_t* parents, int64_t n, int64_t tree_words,
                                     int64_t* words);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_SERVING_H */
