// C ABI of the decoding-step operators (declared in include/convt_decode.h):
// argument checks, the choice of route and split, and the launches.
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>

#include "decode_checks.h"

using namespace convt;

namespace {

convt_status cache_move(const convt_cache_desc *cache, const convt_cache_rows *rows, const void *k, const void *v,
                        const int64_t *slots, const void *k_cache, const void *v_cache, const float *k_scale,
                        const float *v_scale, int write, void *stream) {
    if (!cache || !rows) return CONVT_ERR_INVALID_ARGUMENT;
    const convt_status st = check_cache(*cache);
    if (st != CONVT_OK) return st;
    if (rows->tokens < 0 || rows->tokens > kMaxIndex || rows->tokens * cache->kv_heads > kMaxIndex)
        return CONVT_ERR_INVALID_ARGUMENT;
    if (!strides_ok(rows->k_stride, 2, !write) || !strides_ok(rows->v_stride, 2, !write)) return CONVT_ERR_INVALID_ARGUMENT;
    if (!cache_pointers_ok(*cache, k_cache, v_cache, k_scale, v_scale)) return CONVT_ERR_INVALID_ARGUMENT;
    if (rows->tokens == 0) return CONVT_OK;
    if (!k || !v || !slots) return CONVT_ERR_INVALID_ARGUMENT;
    convt::CacheArgs a{};
    a.k = k;
    a.v = v;
    a.k_cache = const_cast<void *>(k_cache);
    a.v_cache = const_cast<void *>(v_cache);
    a.k_scale = const_cast<float *>(k_scale);
    a.v_scale = const_cast<float *>(v_scale);
    a.slots = slots;
    for (int i = 0; i < 2; ++i) {
        a.row_stride[0][i] = rows->k_stride[i];
        a.row_stride[1][i] = rows->v_stride[i];
    }
    for (int i = 0; i < 3; ++i) {
        a.cache_stride[0][i] = cache->k_stride[i];
        a.cache_stride[1][i] = cache->v_stride[i];
    }
    a.n_slots = cache->n_pages * cache->page_size;
    a.tokens = rows->tokens;
    a.kv_heads = cache->kv_heads;
    a.page_size = cache->page_size;
    a.head_dim = cache->head_dim;
    a.div_heads = convt::divisor_of((uint32_t)cache->kv_heads);
    a.div_page = convt::divisor_of((uint32_t)cache->page_size);
    if (write && a.n_slots == 0) return CONVT_OK;  // no slot is in the cache
    return device_status(convt::launch_cache(a, cache->dtype, cache->quantised, write, (hipStream_t)stream));
}

// Whether the MFMA attention kernel serves a problem (pointers apart).
bool attend_mfma_serves(const convt_attend_problem &p) {
    const convt_cache_desc &c = p.cache;
    if (c.dtype == CONVT_DTYPE_F32 || c.head_dim % 16 != 0 || c.head_dim > 256 || c.page_size % 16 != 0) return false;
    const int64_t piece = c.quantised ? 16 : 8;  // elements in 16 bytes
    for (int i = 0; i < 3; ++i)
        if (c.k_stride[i] % piece != 0 || c.v_stride[i] % piece != 0) return false;
    return p.q_stride[0] % 8 == 0 && p.q_stride[1] % 8 == 0;
}

convt_status attend_check(const convt_attend_problem *p, convt_attend_info *info) {
    if (!p) return CONVT_ERR_INVALID_ARGUMENT;
    const convt_cache_desc &c = p->cache;
    const convt_status st = check_cache(c);
    if (st != CONVT_OK) return st;
    if (p->batch < 0 || p->heads < 1 || p->heads % c.kv_heads != 0) return CONVT_ERR_INVALID_ARGUMENT;
    if ((int64_t)p->batch * p->heads > kMaxBlocks) return CONVT_ERR_UNSUPPORTED;
    if (p->table_width < 0 || p->table_width > kMaxIndex) return CONVT_ERR_INVALID_ARGUMENT;
    if (p->batch > 1 && !row_stride_ok(p->table_stride, p->table_width, true)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p->max_length < 0 || p->max_length > kMaxIndex - 4096 || p->max_length > p->table_width * c.page_size)
        return CONVT_ERR_INVALID_ARGUMENT;
    if (!strides_ok(p->q_stride, 2, 0) || !strides_ok(p->out_stride, 2)) return CONVT_ERR_INVALID_ARGUMENT;
    if (!isfinite(p->scale)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p->route < CONVT_ATTEND_AUTO || p->route > CONVT_ATTEND_MFMA) return CONVT_ERR_INVALID_ARGUMENT;
    const bool mfma = attend_mfma_serves(*p);
    if (p->route == CONVT_ATTEND_MFMA && !mfma) return CONVT_ERR_UNSUPPORTED;
    info->route = mfma && p->route != CONVT_ATTEND_DIRECT ? CONVT_ATTEND_MFMA : CONVT_ATTEND_DIRECT;
    // Parts of the length axis: as many blocks as the card holds at once (256
    // CUs with 4, 3 or 1 of them, by the registers a head dimension takes) if
    // every stream had max_length; parts of at least 128 tokens, a step of each
    // wave. Streams differ, so parts are at most 512 tokens, that the blocks
    // of a long stream need not run after all others have ended, but 1/64 of
    // a long axis (up to 2048), where the join of more parts would cost more.
    // Measured, us (parts of 128, 256, 512, 1024, 2048 tokens): 32 ragged streams
    // up to 4096 x 8 kv heads, e4m3: 50, 41, 38, 37, 40; 4 streams of 100-131 K, bf16:
    // 415, 369, 347, 334, 326; one stream of 60 K, one kv head of 256: 39, 27,
    // 25, 32, 49; one of 3000, two heads, e4m3: 8.7, 9.3, 10.8, 14.4, 21.9.
    const int64_t items = (int64_t)p->batch * c.kv_heads;
    const int64_t slots = 256 * (c.head_dim <= 64 ? 4 : c.head_dim <= 128 ? 3 : 1);
    const int64_t longest = p->max_length / 64 < 512 ? 512 : p->max_length / 64 > 2048 ? 2048 : p->max_length / 64;
    int64_t chunk = p->max_length / 128 * items / slots;  // steps of 128 tokens
    chunk = chunk < 16 ? (chunk + 1) * 128 : 2048;
    if (chunk > longest) chunk = (longest + 127) / 128 * 128;
    // What one block reads in about the time of the second launch stays one
    // part: 512 tokens of two kv heads, e4m3, 7.2 us in one launch, 7.4 in two
    // (8.0 and 12.3 called from Python); 32 streams of 512 x 8 heads 9.4 and 13.5.
    const int64_t single = c.head_dim <= 128 ? 512 : 256;
    if (p->max_length <= single) chunk = single;
    int64_t chunks = ceil_div(p->max_length, chunk);
    if (chunks < 1) chunks = 1;
    // the grid's second axis holds the parts
    if (chunks > 32768) {
        chunk = ceil_div(ceil_div(p->max_length, 32768), 128) * 128;
        chunks = ceil_div(p->max_length, chunk);
    }
    info->chunks = (int32_t)chunks;
    info->chunk_tokens = (int32_t)chunk;
    info->workspace_bytes =
        chunks > 1 ? (int64_t)p->batch * p->heads * chunks * (c.head_dim + 2) * (int64_t)sizeof(float) : 0;
    info->reserved = 0;
    return CONVT_OK;
}

// Whether the MFMA product kernel serves a problem (pointers apart).
bool q4_mfma_serves(const convt_q4_problem &p) {
    if (p.dtype == CONVT_DTYPE_F32) return false;
    if (p.group != 32 && p.group != 64 && p.group != 128) return false;
    if (p.rows > (1 << 20)) return false;     // the grid has an axis over rows
    if (p.k / p.group > 2000) return false;   // a tile's scales fit in 64 KB of LDS
    return p.x_stride % (p.x_quantised ? 16 : 8) == 0 || p.rows <= 1;  // rows 16-byte aligned
}

convt_status q4_check(const convt_q4_problem *p, int32_t *route) {
    if (!p) return CONVT_ERR_INVALID_ARGUMENT;
    const convt_status st = check_dtype(p->dtype);
    if (st != CONVT_OK) return st;
    if (!flag(p->x_quantised) || p->reserved != 0) return CONVT_ERR_INVALID_ARGUMENT;
    if (p->rows < 0 || p->n < 0 || p->k < 0 || p->rows > kMaxIndex || p->n > kMaxIndex || p->k > kMaxIndex)
        return CONVT_ERR_INVALID_ARGUMENT;
    if (p->group < 8 || p->group % 8 != 0 || p->k % p->group != 0) return CONVT_ERR_INVALID_ARGUMENT;
    if (p->rows > 1 && (!row_stride_ok(p->x_stride, p->k, true) || !row_stride_ok(p->y_stride, p->n, false)))
        return CONVT_ERR_INVALID_ARGUMENT;
    if (p->route < CONVT_Q4_AUTO || p->route > CONVT_Q4_MFMA) return CONVT_ERR_INVALID_ARGUMENT;
    if ((p->n + 3) / 4 > kMaxBlocks) return CONVT_ERR_UNSUPPORTED;
    const bool mfma = q4_mfma_serves(*p);
    if (p->route == CONVT_Q4_MFMA && !mfma) return CONVT_ERR_UNSUPPORTED;
    *route = mfma && p->route != CONVT_Q4_DIRECT ? CONVT_Q4_MFMA : CONVT_Q4_DIRECT;
    return CONVT_OK;
}

}  // namespace

extern "C" {

convt_status convt_rms_norm(const convt_rms_norm_problem *problem, const void *x, const void *weight,
                            const void *residual, void *y, float *scale, void *residual_out, void *stream) {
    if (!problem) return CONVT_ERR_INVALID_ARGUMENT;
    const convt_rms_norm_problem &p = *problem;
    const convt_status st = check_dtype(p.dtype);
    if (st != CONVT_OK) return st;
    if (!flag(p.has_residual) || !flag(p.quantise)) return CONVT_ERR_INVALID_ARGUMENT;
    if (!(p.eps >= 0.0f) || !isfinite(p.eps)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.rows < 0 || p.rows > kMaxIndex || p.width < 1 || p.width > ((int64_t)1 << 24)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.rows > 1) {
        if (!row_stride_ok(p.x_stride, p.width, true) || !row_stride_ok(p.y_stride, p.width, false))
            return CONVT_ERR_INVALID_ARGUMENT;
        if (p.has_residual && (!row_stride_ok(p.residual_stride, p.width, true) ||
                               !row_stride_ok(p.residual_out_stride, p.width, false)))
            return CONVT_ERR_INVALID_ARGUMENT;
    }
    if (p.has_residual ? 0 : (residual || residual_out)) return CONVT_ERR_INVALID_ARGUMENT;
    if (!p.quantise && scale) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.rows == 0) return CONVT_OK;
    if (!x || !weight || !y) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.has_residual && (!residual || !residual_out)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.quantise && !scale) return CONVT_ERR_INVALID_ARGUMENT;
    return device_status(
        convt::launch_rms_norm(p, x, weight, residual, y, scale, residual_out, (hipStream_t)stream));
}

convt_status convt_cache_write(const convt_cache_desc *cache, const convt_cache_rows *rows, const void *k,
                               const void *v, const int64_t *slots, void *k_cache, void *v_cache, float *k_scale,
                               float *v_scale, void *stream) {
    return cache_move(cache, rows, k, v, slots, k_cache, v_cache, k_scale, v_scale, 1, stream);
}

convt_status convt_cache_read(const convt_cache_desc *cache, const convt_cache_rows *rows, const void *k_cache,
                              const void *v_cache, const float *k_scale, const float *v_scale, const int64_t *slots,
                              void *k, void *v, void *stream) {
    return cache_move(cache, rows, k, v, slots, k_cache, v_cache, k_scale, v_scale, 0, stream);
}

convt_status convt_attend_query(const convt_attend_problem *problem, convt_attend_info *info) {
    if (!info) return CONVT_ERR_INVALID_ARGUMENT;
    return attend_check(problem, info);
}

convt_status convt_attend(const convt_attend_problem *problem, const void *q, const void *k_cache,
                          const void *v_cache, const float *k_scale, const float *v_scale, const int32_t *page_table,
                          const int32_t *lengths, void *out, float *lse, void *workspace, void *stream) {
    convt_attend_info info;
    const convt_status st = attend_check(problem, &info);
    if (st != CONVT_OK) return st;
    const convt_attend_problem &p = *problem;
    const convt_cache_desc &c = p.cache;
    if (!cache_pointers_ok(c, k_cache, v_cache, k_scale, v_scale)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.batch == 0) return CONVT_OK;
    if (!q || !out || !lengths || (p.table_width > 0 && !page_table)) return CONVT_ERR_INVALID_ARGUMENT;
    if (info.workspace_bytes > 0 && (!workspace || !aligned(workspace, 16))) return CONVT_ERR_INVALID_ARGUMENT;
    convt::AttendArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.page_table = page_table;
    a.lengths = lengths;
    a.out = out;
    a.lse = lse;
    a.part_o = (float *)workspace;
    a.part_ml = (float *)workspace + (int64_t)p.batch * p.heads * info.chunks * c.head_dim;
    for (int i = 0; i < 2; ++i) {
        a.q_stride[i] = p.q_stride[i];
        a.out_stride[i] = p.out_stride[i];
    }
    for (int i = 0; i < 3; ++i) {
        a.k_stride[i] = c.k_stride[i];
        a.v_stride[i] = c.v_stride[i];
    }
    a.table_stride = p.table_stride;
    a.n_pages = c.n_pages;
    a.batch = p.batch;
    a.heads = p.heads;
    a.kv_heads = c.kv_heads;
    a.share = p.heads / c.kv_heads;
    a.head_dim = c.head_dim;
    a.page_size = c.page_size;
    // without pages there is nothing to read
    a.max_length = c.n_pages > 0 ? (int32_t)p.max_length : 0;
    a.chunks = info.chunks;
    a.chunk_tokens = info.chunk_tokens;
    a.scale_log2e = (float)((double)p.scale * 1.4426950408889634074);
    a.div_page = convt::divisor_of((uint32_t)c.page_size);
    a.div_heads = convt::divisor_of((uint32_t)p.heads);
    const hipStream_t s = (hipStream_t)stream;
    const bool mfma = info.route == CONVT_ATTEND_MFMA && aligned(q, 16) && aligned(k_cache, 16) &&
                      aligned(v_cache, 16) && aligned(k_scale, 16) && aligned(v_scale, 16);
    hipError_t e = mfma ? convt::launch_attend_mfma(a, c.dtype, c.quantised, s)
                        : convt::launch_attend_direct(a, c.dtype, c.quantised, s);
    if (e == hipSuccess && a.chunks > 1) e = convt::launch_attend_join(a, c.dtype, s);
    return device_status(e);
}

convt_status convt_q4_query(const convt_q4_problem *problem, int32_t *route) {
    if (!route) return CONVT_ERR_INVALID_ARGUMENT;
    return q4_check(problem, route);
}

convt_status convt_q4_matvec(const convt_q4_problem *problem, const void *x, const float *x_scale, const void *w,
                             const void *scales, void *y, void *stream) {
    int32_t route;
    const convt_status st = q4_check(problem, &route);
    if (st != CONVT_OK) return st;
    const convt_q4_problem &p = *problem;
    if (!p.x_quantised && x_scale) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.rows == 0 || p.n == 0) return CONVT_OK;
    if (!y || (p.x_quantised && !x_scale)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.k > 0 && (!x || !w || !scales)) return CONVT_ERR_INVALID_ARGUMENT;
    const hipStream_t s = (hipStream_t)stream;
    const bool mfma = route == CONVT_Q4_MFMA && aligned(x, 16) && aligned(w, 16);
    return device_status(mfma ? convt::launch_q4_mfma(p, x, x_scale, w, scales, y, s)
                              : convt::launch_q4_direct(p, x, x_scale, w, scales, y, s));
}

}  // extern "C"
