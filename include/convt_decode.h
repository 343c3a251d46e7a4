/*
 * convt_decode.h — C ABI of the decoding-step operators of libconvt (gfx950).
 *
 * A decoder-only model that generates the latent frames an upsampler takes
 * works one frame (token) per stream at a time. These operators are the
 * memory-bound part of that step: the residual addition and root-mean-square
 * norm, products with 4-bit weights, the paged key-value cache, and the
 * attention of the new token over it. They serve inference; none has a
 * backward pass.
 *
 * Conventions are those of convt.h: every entry point returns a
 * convt_status; argument errors are found on the host before anything is
 * enqueued; device work is asynchronous on `stream`, a stream of the current
 * device, where all buffers lie; the caller owns every buffer and the
 * workspace; nothing is kept after a call returns and no entry point
 * allocates memory, so every call may be captured into a graph.
 * CONVT_ERR_INVALID_ARGUMENT reports a value, shape, stride, alignment or
 * missing pointer that breaks a rule below, CONVT_ERR_UNSUPPORTED a
 * well-formed request that is not computed. Element types are CONVT_DTYPE_F32,
 * _BF16 and _F16; sums, softmax statistics and scales are float32.
 *
 * 8-bit values are OCP e4m3 (4 exponent bits, 3 mantissa bits, largest finite
 * value 448, no infinities). A quantised row r (a row of a norm's output, or
 * one token's key or value of one head) is held as e4m3 codes q and one
 * float32 scale s with r ~ q * s:
 *     s = max(max|r| / 448, 2^-126),   q = round_to_nearest_even(r * (1/s)).
 * A row holding a NaN has s = NaN, one holding an infinity s = infinity and
 * codes that are 0 or NaN: both read back as NaN in every place.
 *
 * Problem structs are zero-initialised by the caller and then filled;
 * fields named reserved must be 0. Strides count elements; those of what a call
 * only reads may be 0 (a repeated row), others are at least 1, none above 2^40.
 */
#ifndef CONVT_DECODE_H
#define CONVT_DECODE_H

#include <stdint.h>

#include "convt.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Residual addition and root-mean-square norm:
 *     h[r, i] = x[r, i] + residual[r, i]          (x alone without a residual)
 *     y[r, i] = h[r, i] / sqrt(mean_i h[r, i]^2 + eps) * weight[i]
 * in float32 throughout (a row whose sum of squares is not finite there, |h| of
 * some 1.8e19, gives 0, or NaN where h is infinite); residual_out receives h
 * rounded to the element type (the norm itself uses h before that rounding). y
 * is rounded to the element type, or, with quantise = 1, quantised per row: y
 * then holds e4m3 codes (bytes) and scale one float32 per row.
 * rows >= 0, width in 1 .. 2^24; row strides >= width, those of x and residual
 * also 0 (read only when rows > 1). residual and residual_out are required iff
 * has_residual; scale iff quantise. residual_out may be residual or x itself,
 * and y may be x or residual when not quantised and the strides agree (each
 * element is read before its place is written); otherwise outputs overlap no
 * input.
 */
typedef struct convt_rms_norm_problem {
    int64_t rows, width;
    int64_t x_stride, residual_stride, y_stride, residual_out_stride;
    int32_t dtype;          /* convt_dtype of x, weight, residual, residual_out and unquantised y */
    int32_t has_residual;   /* 0 or 1 */
    int32_t quantise;       /* 0 or 1 */
    float eps;              /* >= 0, finite */
} convt_rms_norm_problem;

convt_status convt_rms_norm(const convt_rms_norm_problem *problem, const void *x, const void *weight,
                            const void *residual, void *y, float *scale, void *residual_out,
                            void *stream);

/*
 * A paged key-value cache: pages of page_size tokens. Keys and values are two
 * arrays indexed [page][kv head][token of the page][dim] through strides
 * (elements; the last is 1, so a cache stored [page][token][head][dim] is
 * passed with its strides exchanged). Unquantised caches hold the element
 * type; quantised ones e4m3 codes, with k_scale and v_scale contiguous
 * float32 arrays [n_pages][kv_heads][page_size]. Slot s = page * page_size +
 * token names one token's place.
 * n_pages >= 0, kv_heads >= 1, page_size >= 1, 1 <= head_dim <= 512,
 * n_pages * page_size < 2^31; strides >= 1.
 */
typedef struct convt_cache_desc {
    int64_t n_pages;
    int64_t k_stride[3], v_stride[3];  /* page, head, token */
    int32_t kv_heads, page_size, head_dim;
    int32_t dtype;          /* element type (what k and v are given and read in) */
    int32_t quantised;      /* 0: the cache holds dtype; 1: e4m3 and scales */
    int32_t reserved;
} convt_cache_desc;

/*
 * Write tokens' keys and values into the cache: k and v are [tokens][kv_heads]
 * [head_dim] of the element type with the given token and head strides (the
 * last is 1), slots[t] the slot of token t. Tokens whose slot is negative or
 * not below n_pages * page_size are not written. The slots of a call that are
 * written differ: a place named twice may be left with parts of both tokens
 * (one's codes, the other's scale); other places are as they should be.
 * tokens >= 0; tokens * kv_heads < 2^31.
 */
typedef struct convt_cache_rows {
    int64_t tokens;
    int64_t k_stride[2], v_stride[2];  /* token, head */
} convt_cache_rows;

convt_status convt_cache_write(const convt_cache_desc *cache, const convt_cache_rows *rows, const void *k,
                               const void *v, const int64_t *slots, void *k_cache, void *v_cache,
                               float *k_scale, float *v_scale, void *stream);

/*
 * The inverse: read the tokens at `slots` into k and v (element type; codes
 * times scales in float32, rounded once). Rows of a slot outside the cache
 * become zeros.
 */
convt_status convt_cache_read(const convt_cache_desc *cache, const convt_cache_rows *rows, const void *k_cache,
                              const void *v_cache, const float *k_scale, const float *v_scale,
                              const int64_t *slots, void *k, void *v, void *stream);

/*
 * Attention of one new token per stream over the cache:
 *     out[b, h] = sum_t p[t] V[t],  p = softmax over t < length[b] of
 *                 scale * <q[b, h], K[t]>,
 * K and V the tokens of kv head h / (heads / kv_heads) in the pages
 * page_table[b][t / page_size]. The softmax is in float32. lse, if wanted,
 * receives the natural logarithm of the sum of exponentials (float32
 * [batch][heads]), for joining with attention over other keys. A stream that
 * sees nothing (length <= 0) gets out = 0 and lse = -infinity. Lengths above
 * max_length are cut to it; tokens of a page id outside 0 .. n_pages - 1 are
 * left out. Nothing past a stream's length is read into the result, whatever
 * it holds. An infinite or NaN value that is seen makes its dim of the result
 * so, as the formula does; a weight too small to be held (2^-126 of the
 * largest, 2^-40 over a float16 cache on the matrix cores) times an infinite
 * value is NaN.
 *
 * max_length bounds the lengths the call handles: at most table_width *
 * page_size, and below 2^31 - 4096. The length axis is cut into chunks that are computed by different
 * blocks and joined by a second kernel through the workspace; with one chunk
 * there is one kernel and no workspace.
 *
 * heads is a multiple of cache.kv_heads, batch * heads below 2^24; q and out have the given batch and
 * head strides (the last is 1), page_table int32 [batch][table_width] with
 * table_stride (0, or at least table_width) between its rows, lengths int32
 * [batch]. scale is finite.
 * Routes: ATTEND_MFMA (two-byte types, head_dim a multiple of 16 and at most
 * 256, page_size a multiple of 16, 16-byte aligned cache rows) on the matrix
 * cores; ATTEND_DIRECT for everything else. route = CONVT_ATTEND_AUTO picks;
 * a forced ATTEND_MFMA that cannot serve is CONVT_ERR_UNSUPPORTED. (The
 * route is fixed by the problem; a cache or query pointer that is not 16-byte
 * aligned runs the direct kernel instead, same result within rounding.)
 */
typedef enum convt_attend_route {
    CONVT_ATTEND_AUTO = 0,
    CONVT_ATTEND_DIRECT = 1,
    CONVT_ATTEND_MFMA = 2
} convt_attend_route;

typedef struct convt_attend_problem {
    convt_cache_desc cache;
    int64_t max_length;
    int64_t q_stride[2], out_stride[2];  /* batch, head */
    int64_t table_width, table_stride;
    int32_t batch, heads;
    int32_t route;          /* convt_attend_route */
    float scale;
} convt_attend_problem;

typedef struct convt_attend_info {
    int64_t workspace_bytes;
    int32_t route;          /* the route chosen */
    int32_t chunks;         /* parts the length axis is cut into */
    int32_t chunk_tokens;   /* tokens of a part */
    int32_t reserved;
} convt_attend_info;

/* Validate a problem and report its route and workspace. Host only. */
convt_status convt_attend_query(const convt_attend_problem *problem, convt_attend_info *info);

/* workspace: workspace_bytes bytes, 16-byte aligned (NULL allowed when 0), not
 * in use by another call. lse may be NULL. */
convt_status convt_attend(const convt_attend_problem *problem, const void *q, const void *k_cache,
                          const void *v_cache, const float *k_scale, const float *v_scale,
                          const int32_t *page_table, const int32_t *lengths, void *out, float *lse,
                          void *workspace, void *stream);

/*
 * Products of a few rows with 4-bit weights:
 *     y[m, n] = x_scale[m] * sum_g scales[n, g] * sum_{k in group g} x[m, k] * (w[n, k] - 8)
 * w: [n][k / 2] bytes, the even k in the low four bits, values 0 .. 15 that
 * stand for -8 .. 7 (a row of x that holds an infinity or NaN gives results that
 * are not finite either); scales [n][k / group] of the element type; both
 * contiguous. x is [rows][k] of the element type, or, with x_quantised = 1,
 * e4m3 codes with x_scale float32 [rows] (the norm's quantised output;
 * x_scale is left out otherwise). y is [rows][n] of the element type. Sums in
 * float32, one rounding. On the matrix cores they run over x * w and 8 x, so
 * their roundings are those of terms of up to 15 |x| (weights of 0 alone give
 * about 2^-24 of sum 8 |x|, not always 0).
 * rows >= 0, n >= 0, k >= 0; group a multiple of 8 that divides k; row
 * strides of x >= k or 0 and of y >= n (read only when rows > 1); rows and k below
 * 2^31, n at most 2^26 - 4.
 * Routes: Q4_MFMA (two-byte types, group 32, 64 or 128, w and x rows 16-byte
 * aligned) on the matrix cores; Q4_DIRECT for everything
 * else, also at run time for pointers not so aligned.
 */
typedef enum convt_q4_route {
    CONVT_Q4_AUTO = 0,
    CONVT_Q4_DIRECT = 1,
    CONVT_Q4_MFMA = 2
} convt_q4_route;

typedef struct convt_q4_problem {
    int64_t rows, n, k, group;
    int64_t x_stride, y_stride;
    int32_t dtype;          /* convt_dtype of scales, y and unquantised x */
    int32_t x_quantised;    /* 0 or 1 */
    int32_t route;          /* convt_q4_route */
    int32_t reserved;
} convt_q4_problem;

/* Validate a problem and report its route (convt_q4_route). Host only. */
convt_status convt_q4_query(const convt_q4_problem *problem, int32_t *route);

convt_status convt_q4_matvec(const convt_q4_problem *problem, const void *x, const float *x_scale,
                             const void *w, const void *scales, void *y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVT_DECODE_H */
