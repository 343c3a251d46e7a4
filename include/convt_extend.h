/*
 * convt_extend.h — C ABI of the operators of steps with several new tokens
 * per stream (gfx950): prompts, chunks of prompts, long streams that see a
 * window, and trees of drafted tokens, over the paged cache of convt_decode.h.
 *
 * convt_cache_append rotates queries and keys by their positions and writes
 * keys and values into the cache; convt_window_attend and convt_tree_attend
 * are the attention of the new tokens over it. They serve inference; none has
 * a backward pass.
 *
 * Conventions, the cache's description, the 8-bit format and what a status
 * reports are those of convt_decode.h: checks on the host before anything is
 * enqueued, device work asynchronous on `stream`, caller's buffers, no
 * allocation, every call may be captured into a graph. Strides count
 * elements; those of what a call only reads may be 0, others are at least 1,
 * none above 2^40.
 */
#ifndef CONVT_EXTEND_H
#define CONVT_EXTEND_H

#include <stdint.h>

#include "convt_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rotary positions and cache write in one pass over tokens t, heads h and
 * the pairs i < rotary_dim / 2 of a head's first rotary_dim dims:
 *     angle[t, i] = positions[t] * inv_freq[i]
 *     (a, b) -> (a cos - b sin, a sin + b cos)
 * with (a, b) dims (i, i + rotary_dim / 2), or (2i, 2i + 1) with interleaved
 * = 1; dims from rotary_dim on stay as they are. q is rotated into q_out
 * (heads = 0: there are no queries), k is rotated and written into the
 * cache at slots[t] as convt_cache_write writes it (quantised after the
 * rotation), v is written there as it is. Tokens whose slot lies outside the
 * cache are not written; their queries are rotated all the same. Slots that
 * are written differ, as in convt_cache_write.
 * The product position * inv_freq and its reduction to a quarter turn are in
 * float64, sine and cosine within some 2^-23, the rotation in float32: the
 * rotated value is rounded once, where it is stored.
 * positions: int64, of any sign, exact up to 2^53 (an angle is off by 2^-52
 * of itself). inv_freq: float32 [rotary_dim / 2].
 * rotary_dim even, 0 .. head_dim; heads >= 0; tokens * (heads + 2 kv_heads)
 * below 2^31. q_out may be q itself if the strides agree; otherwise outputs
 * overlap no input.
 */
typedef struct convt_append_problem {
    convt_cache_desc cache;
    convt_cache_rows rows;               /* tokens, strides of k and v */
    int64_t q_stride[2], q_out_stride[2];  /* token, head (the last is 1) */
    int32_t heads;          /* query heads */
    int32_t rotary_dim;
    int32_t interleaved;    /* 0 or 1 */
    int32_t reserved;
} convt_append_problem;

convt_status convt_cache_append(const convt_append_problem *problem, const void *q, const void *k, const void *v,
                                const int64_t *slots, const int64_t *positions, const float *inv_freq,
                                void *k_cache, void *v_cache, float *k_scale, float *v_scale, void *q_out,
                                void *stream);

/*
 * What the two attentions share. A row is a new token and one of its query
 * heads:
 *     out[row] = sum_t p[t] V[t],  p = softmax over the tokens t that the
 *                row sees of scale * <q[row], K[t]>,
 * K and V of kv head h / (heads / kv_heads) in the pages of the token's stream,
 * page_table[b][t / page_size]. Softmax statistics and sums are float32. lse,
 * if wanted (float32 [tokens][heads]), receives the natural logarithm of the
 * sum of exponentials. A row that sees nothing gets out = 0 and lse =
 * -infinity. Tokens of a page id outside 0 .. n_pages - 1 are left out. What a
 * row does not see changes nothing, whatever it holds; an infinite or NaN value
 * that it sees makes its dim of the result so, a weight too small to be held
 * times an infinite value NaN. A weight below 2^-60 of the row's largest may
 * be lost.
 * Scales of a quantised cache are positive, as its definition gives them
 * (smaller ones count as 2^-126). Those of values may differ by any factor: a
 * row of zeros has its part in the sum of exponentials, and a scale that is not
 * finite makes out NaN, not lse. (One outside 2^-40 .. 2^30 has the sum formed
 * another way, for neighbours that do not see it too: its last bits may differ.)
 *
 * max_length bounds the tokens t < max_length that the call handles: at most
 * table_width * page_size and below 2^31 - 4096. heads is a multiple of
 * cache.kv_heads; the numbers of rows and of streams are below 2^24. q and out are
 * [tokens][heads][head_dim] with the given token and head strides. The
 * axis of t may be cut into parts that are computed by different blocks and
 * joined by a second kernel through the workspace (a close max_length saves
 * room and blocks for parts that no stream reaches). out and lse overlap no
 * input.
 * Routes: EXTEND_MFMA (two-byte types, head_dim a multiple of 16 and at most
 * 256, page_size a multiple of 16, 16-byte aligned rows of cache and q, cache
 * strides below 2^31 elements between pages and 2^25 between tokens) on the
 * matrix cores, EXTEND_DIRECT for everything else, also at run time for
 * pointers not so aligned. AUTO picks; a forced MFMA that cannot serve is
 * CONVT_ERR_UNSUPPORTED.
 * EXTEND_DIRECT rounds the result alone. On the matrix cores a weight p is
 * rounded where it meets its value: to float16 over float16 and quantised caches
 * (2^-11 of it), over bfloat16 caches to the sum of two bfloat16 (2^-16) in calls of few
 * rows a stream (new tokens times heads / kv_heads up to 32; ragged streams: on
 * average), and to one (2^-8) in others, whose results are as far off as one
 * more rounding of theirs makes them.
 */
typedef enum convt_extend_route {
    CONVT_EXTEND_AUTO = 0,
    CONVT_EXTEND_DIRECT = 1,
    CONVT_EXTEND_MFMA = 2
} convt_extend_route;

typedef struct convt_extend_info {
    int64_t workspace_bytes;
    int32_t route;          /* the route chosen */
    int32_t chunks;         /* parts the axis of t is cut into, at most */
    int32_t chunk_tokens;   /* tokens of a part of as many */
    int32_t reserved;
} convt_extend_info;

/*
 * Attention of the new tokens of ragged streams, causal, with a window and
 * first tokens that stay visible. Stream b has the rows starts[b] <=
 * i < starts[b + 1] of q (int32 [batch + 1], not decreasing, within 0 ..
 * tokens), which are the last tokens of its lengths[b]: row i has position
 *     p = lengths[b] - (starts[b + 1] - i)
 * and sees the tokens t <= p with t > p - window or t < sinks. starts NULL
 * stands for one new token per stream (tokens = batch). A position below 0 (a
 * stream with more rows than length) sees nothing. Rows that no stream
 * has (behind the last one's) are not written, in out or lse. Lengths above
 * max_length are cut to it.
 * window >= 0; 0 sees every t <= p. sinks >= 0.
 */
typedef struct convt_window_problem {
    convt_cache_desc cache;
    int64_t max_length;
    int64_t tokens;                      /* rows of q and out */
    int64_t q_stride[2], out_stride[2];  /* token, head */
    int64_t table_width, table_stride;
    int64_t window, sinks;
    int32_t batch, heads;
    int32_t ragged;         /* 1: starts is given, 0: one token per stream */
    int32_t route;          /* convt_extend_route */
    float scale;
    int32_t reserved;
} convt_window_problem;

/* Validate a problem and report its route and workspace. Host only. */
convt_status convt_window_query(const convt_window_problem *problem, convt_extend_info *info);

/* workspace: workspace_bytes bytes, 16-byte aligned (NULL allowed when 0), not
 * in use by another call. lse may be NULL. */
convt_status convt_window_attend(const convt_window_problem *problem, const void *q, const void *k_cache,
                                 const void *v_cache, const float *k_scale, const float *v_scale,
                                 const int32_t *page_table, const int32_t *lengths, const int32_t *starts,
                                 void *out, float *lse, void *workspace, void *stream);

/*
 * Attention of `drafts` drafted tokens per stream behind its lengths[b]
 * cached ones: draft i sees every t < lengths[b], and the draft j, which the
 * cache holds at t = lengths[b] + j, if bit j % 64 of tree[b][i][j / 64] is
 * set (so itself, if it has its own bit). Bits of drafts that are not there are
 * ignored. tree: 64-bit words, (drafts + 63) / 64 of them a row, with the given
 * strides (batch, draft; 0 repeats). lengths below 0 count as 0, t from
 * max_length on are left out. q and out are [batch][drafts][heads][head_dim].
 * drafts in 1 .. 1024.
 */
typedef struct convt_tree_problem {
    convt_cache_desc cache;
    int64_t max_length;
    int64_t q_stride[3], out_stride[3];  /* batch, draft, head */
    int64_t tree_stride[2];              /* batch, draft, in words */
    int64_t table_width, table_stride;
    int32_t batch, drafts, heads;
    int32_t route;          /* convt_extend_route */
    float scale;
    int32_t reserved;
} convt_tree_problem;

/* Validate a problem and report its route and workspace. Host only. */
convt_status convt_tree_query(const convt_tree_problem *problem, convt_extend_info *info);

convt_status convt_tree_attend(const convt_tree_problem *problem, const void *q, const void *k_cache,
                               const void *v_cache, const float *k_scale, const float *v_scale,
                               const int32_t *page_table, const int32_t *lengths, const uint64_t *tree, void *out,
                               float *lse, void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVT_EXTEND_H */
