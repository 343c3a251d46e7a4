// C ABI of the operators of several new tokens per stream (declared in
// include/convt_extend.h): argument checks, the choice of route and split, and
// the launches.
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>

#include "decode_checks.h"
#include "extend.h"

using namespace convt;

namespace {

// Whether the matrix-core kernel serves a cache and q strides (pointers apart).
bool mfma_serves(const convt_cache_desc &c, const int64_t *q_stride, int n) {
    if (c.dtype == CONVT_DTYPE_F32 || c.head_dim % 16 != 0 || c.head_dim > 256 || c.page_size % 16 != 0) return false;
    const int64_t piece = c.quantised ? 16 : 8;  // elements in 16 bytes
    for (int i = 0; i < 3; ++i)
        if (c.k_stride[i] % piece != 0 || c.v_stride[i] % piece != 0) return false;
    // the kernel's factors of a tile's offset, and a lane's bytes within 16 tokens, have 32 bits
    if (c.k_stride[0] >> 31 || c.v_stride[0] >> 31 || c.k_stride[2] >> 25 || c.v_stride[2] >> 25) return false;
    if (((int64_t)c.kv_heads * c.page_size) >> 31) return false;
    for (int i = 0; i < n; ++i)
        if (q_stride[i] % 8 != 0) return false;
    return true;
}

// The form of the matrix-core kernel and its tiles for streams of `each` new
// tokens (ragged ones: on average).
struct Shape {
    ExtendForm form;
    int64_t block_tokens, head_tiles, stream_tiles, tiles;
    int64_t slots, least;  // blocks that the card holds at once, tokens of a part at least
};
Shape shape_of(ExtendForm form, int64_t batch, int64_t tokens, int64_t each, bool ragged, int64_t share, int32_t head_dim) {
    Shape s;
    s.form = form;
    const int64_t rows = form == ExtendForm::kKeys ? 32 : form == ExtendForm::kRows128 ? 128 : 256;
    s.block_tokens = share >= rows ? 1 : rows / share;
    s.head_tiles = ceil_div(share, rows);
    s.stream_tiles = ragged ? 0 : ceil_div(each, s.block_tokens);
    // ragged: every stream with rows may end in a tile of its own
    s.tiles = ragged ? tokens / s.block_tokens + (batch < tokens ? batch : tokens) : batch * s.stream_tiles;
    s.slots = 256 * (head_dim <= 128 && form != ExtendForm::kRows256 ? 2 : 1);
    s.least = form == ExtendForm::kKeys ? 128 : 512;
    return s;
}
// Rows of a stream that fit in 32 share their tokens among a block's waves; more go 128 or 256 to a block
// (above 128 dims 128: a SIMD has the registers of one wave then, 4 a block). Measured, us, the form for few
// rows and 128 rows, 4 heads sharing a kv head, 8 of these: trees of 8 drafts over 16 x 4096: 52, 52;
// of 16: 59, 57; of 25 over ragged ones: 67, 51; one token in a window of 4096, 64 streams: 108, 160. 256 rows a block are faster
// where blocks fill the card twice, or will do once the axis is cut, since it is long
// against the new tokens; else the card's last blocks take too long. Measured, us, 128 and 256 rows, 32 / 8 heads of
// 128, bf16: prompts of 512: 22, 27; 2048: 68, 66; 4096: 179, 155; 5 ragged chunks of 500 to 1000 in a
// window of 513 (20 / 4 heads of 96): 53, 62; trees of 64 drafts over 2 x 131 K: 358, 320; 512 new ones of 16384: 174, 152.
Shape pick_shape(int64_t batch, int64_t tokens, int64_t each, bool ragged, int64_t heads, int64_t kv_heads, int32_t head_dim, int64_t longest) {
    const int64_t share = heads / kv_heads;
    if (each * share <= 32) return shape_of(ExtendForm::kKeys, batch, tokens, each, ragged, share, head_dim);
    if (each * share > 128 && head_dim <= 128) {
        const Shape s = shape_of(ExtendForm::kRows256, batch, tokens, each, ragged, share, head_dim);
        const int64_t blocks = s.tiles * s.head_tiles * kv_heads;
        if (blocks >= 2 * s.slots || (longest / 4 >= each && blocks * (longest / s.least) >= s.slots)) return s;
    }
    Shape s = shape_of(ExtendForm::kRows128, batch, tokens, each, ragged, share, head_dim);
    if (longest / 4 >= each) s.least = 256;
    return s;
}

// What window and tree problems are checked for alike, and the info of one
// whose rows see at most `longest` tokens. limited: a window limits them.
convt_status extend_check(const convt_cache_desc &c, int64_t max_length, int64_t batch, int64_t tokens, int64_t each, bool ragged,
                          int64_t heads, const int64_t *q_stride, const int64_t *out_stride, int n_strides, int64_t table_width,
                          int64_t table_stride, int32_t route, float scale, int64_t longest, bool limited, convt_extend_info *info,
                          Shape *shape) {
    const convt_status st = check_cache(c);
    if (st != CONVT_OK) return st;
    if (batch < 0 || tokens < 0 || heads < 1 || heads % c.kv_heads != 0) return CONVT_ERR_INVALID_ARGUMENT;
    // (streams without rows take no blocks, but blocks go through all of them, with 32-bit indexes)
    if (batch > kMaxBlocks || tokens > kMaxBlocks || tokens * heads > kMaxBlocks) return CONVT_ERR_UNSUPPORTED;
    if (table_width < 0 || table_width > kMaxIndex) return CONVT_ERR_INVALID_ARGUMENT;
    if (batch > 1 && !row_stride_ok(table_stride, table_width, true)) return CONVT_ERR_INVALID_ARGUMENT;
    if (max_length < 0 || max_length > kMaxIndex - 4096 || max_length > table_width * c.page_size)
        return CONVT_ERR_INVALID_ARGUMENT;
    if (!strides_ok(q_stride, n_strides, 0) || !strides_ok(out_stride, n_strides)) return CONVT_ERR_INVALID_ARGUMENT;
    if (!isfinite(scale)) return CONVT_ERR_INVALID_ARGUMENT;
    if (route < CONVT_EXTEND_AUTO || route > CONVT_EXTEND_MFMA) return CONVT_ERR_INVALID_ARGUMENT;
    *shape = pick_shape(batch, tokens, each, ragged, heads, c.kv_heads, c.head_dim, longest);
    const int64_t blocks = shape->tiles * shape->head_tiles * c.kv_heads;
    const bool mfma = mfma_serves(c, q_stride, n_strides) && blocks <= kMaxBlocks;
    if (route == CONVT_EXTEND_MFMA && !mfma) return CONVT_ERR_UNSUPPORTED;
    info->route = mfma && route != CONVT_EXTEND_DIRECT ? CONVT_EXTEND_MFMA : CONVT_EXTEND_DIRECT;
    const int64_t rows = tokens * heads;
    int64_t chunks, least;
    if (info->route == CONVT_EXTEND_MFMA) {
        // Parts at most: the kernel takes as many of them as the streams' real lengths make worth while, so
        // that the card is full once. Without a window streams may differ: up to three times as many parts
        // for the long ones. Blocks that fill the card twice need none. Measured, us (1, 2, 3, 4, 6, 8
        // parts): 16 ragged streams up to 4096, 25 drafts: 134, 80, 72, 62, 51, 64; 4 of 2100 to 8000, 512
        // new tokens: 277, 265, 227, 254, 257, 258; 64 in a window of 4096, one new token: 110, 117, 122, 126, 133, 141.
        // At most as many, twice, three, four times as many as fill the card: the 16 streams: 66, 54, 54, 54; 6 chunks of 300 over
        // 300 to 12000, e4m3: 306, 308, 276, 276; 8 of 256 over 256 to 16384, bf16: 416, 321, 323, 319; 32 trees of 8 over 1 to
        // 8192, e4m3: 87, 73, 73, 73; but 8 of 64 over 1 to 8192, bf16: 76, 94, 95, 94, and of 16 over 1 to 16384: 81, 97, 98, 98.
        // Up to 512 tokens one part: the join's launch takes as long (260 tokens: 8.8 us in one). Parts of few rows have
        // 128 tokens at least, a step of each wave; of many 256, or 512 where the rows are most of the tokens.
        // (1, 2, 4, 8, 16 parts) one token of 1024: 19.0, 16.7, 13.9, 12.9, -; of 4096: 54, 35, 23, 18, 16; 16
        // drafts of 2048: 52, 33, 22, 18.5, 16.8; a prompt of 512: 22, 25, 26.
        if (blocks == 0 || blocks >= 2 * shape->slots || longest <= 512) chunks = 1;
        else if (limited) chunks = shape->slots / blocks;
        else chunks = ceil_div((batch < 3 ? batch : 3) * shape->slots, blocks);
        least = shape->least;
    } else {
        chunks = rows > 0 ? 2048 / rows : 1;
        least = 2048;
    }
    if (chunks > longest / least) chunks = longest / least;
    if (blocks > 0 && chunks > kMaxBlocks / blocks) chunks = kMaxBlocks / blocks;
    if (chunks < 1) chunks = 1;
    const int64_t chunk = ceil_div(ceil_div(longest > 0 ? longest : 1, chunks), 64) * 64;
    chunks = longest > 0 ? ceil_div(longest, chunk) : 1;
    info->chunks = (int32_t)chunks;
    info->chunk_tokens = (int32_t)chunk;
    info->workspace_bytes = chunks > 1 ? rows * (chunks * (c.head_dim + 2) + 1) * (int64_t)sizeof(float) : 0;
    info->reserved = 0;
    return CONVT_OK;
}

convt_status window_check(const convt_window_problem *p, convt_extend_info *info, Shape *shape) {
    if (!p) return CONVT_ERR_INVALID_ARGUMENT;
    if (!flag(p->ragged) || p->reserved != 0 || p->window < 0 || p->sinks < 0) return CONVT_ERR_INVALID_ARGUMENT;
    if (!p->ragged && p->tokens != p->batch) return CONVT_ERR_INVALID_ARGUMENT;
    const bool limited = p->window > 0 && p->window < p->max_length && p->sinks < p->max_length - p->window;
    const int64_t each = p->ragged && p->batch > 0 ? ceil_div(p->tokens, p->batch) : 1;
    return extend_check(p->cache, p->max_length, p->batch, p->tokens, each, p->ragged != 0, p->heads, p->q_stride, p->out_stride, 2,
                        p->table_width, p->table_stride, p->route, p->scale, limited ? p->window + p->sinks : p->max_length, limited,
                        info, shape);
}

convt_status tree_check(const convt_tree_problem *p, convt_extend_info *info, Shape *shape) {
    if (!p) return CONVT_ERR_INVALID_ARGUMENT;
    if (p->reserved != 0 || p->drafts < 1 || p->batch < 0) return CONVT_ERR_INVALID_ARGUMENT;
    if (p->drafts > 1024) return CONVT_ERR_UNSUPPORTED;
    if (!strides_ok(p->tree_stride, 2, 0)) return CONVT_ERR_INVALID_ARGUMENT;
    return extend_check(p->cache, p->max_length, p->batch, (int64_t)p->batch * p->drafts, p->drafts, false, p->heads, p->q_stride,
                        p->out_stride, 3, p->table_width, p->table_stride, p->route, p->scale, p->max_length, false, info, shape);
}

// The fields that both problems fill alike.
ExtendArgs common_args(const convt_cache_desc &c, const convt_extend_info &info, int64_t tokens, int64_t heads, int64_t max_length,
                       float scale, const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                       const float *v_scale, const int32_t *page_table, const int32_t *lengths, void *out, float *lse,
                       void *workspace) {
    ExtendArgs a{};
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
    a.part_ml = (float *)workspace + tokens * heads * info.chunks * c.head_dim;
    a.part_count = (int32_t *)((float *)workspace + tokens * heads * info.chunks * (c.head_dim + 2));
    for (int i = 0; i < 3; ++i) {
        a.k_stride[i] = c.k_stride[i];
        a.v_stride[i] = c.v_stride[i];
    }
    a.n_pages = c.n_pages;
    a.tokens = (int32_t)tokens;
    a.heads = (int32_t)heads;
    a.kv_heads = c.kv_heads;
    a.share = (int32_t)(heads / c.kv_heads);
    a.head_dim = c.head_dim;
    a.page_size = c.page_size;
    // without pages there is nothing to read
    a.max_length = c.n_pages > 0 ? (int32_t)max_length : 0;
    a.chunks = info.chunks;
    a.chunk_tokens = info.chunk_tokens;
    a.scale_log2e = (float)((double)scale * 1.4426950408889634074);
    a.div_page = divisor_of((uint32_t)c.page_size);
    a.div_heads = divisor_of((uint32_t)heads);
    a.div_drafts = divisor_of(1);
    return a;
}

convt_status launch(const ExtendArgs &a, const convt_cache_desc &c, const convt_extend_info &info, const Shape &shape, hipStream_t s) {
    const bool mfma = info.route == CONVT_EXTEND_MFMA && aligned(a.q, 16) && aligned(a.k_cache, 16) && aligned(a.v_cache, 16);
    hipError_t e;
    if (mfma) {
        ExtendTiles t;
        t.form = shape.form;
        t.block_tokens = (int32_t)shape.block_tokens;
        t.head_tiles = (int32_t)shape.head_tiles;
        t.stream_tiles = (int32_t)shape.stream_tiles;
        t.tiles = (int32_t)shape.tiles;
        t.slots = (int32_t)shape.slots;
        t.least = (int32_t)shape.least;
        t.div_kv = divisor_of((uint32_t)a.kv_heads);
        t.div_tiles = divisor_of((uint32_t)t.tiles);
        t.div_block_tokens = divisor_of((uint32_t)t.block_tokens);
        t.div_head_tiles = divisor_of((uint32_t)t.head_tiles);
        t.div_stream_tiles = divisor_of((uint32_t)(t.stream_tiles > 0 ? t.stream_tiles : 1));
        if (c.quantised) e = c.dtype == CONVT_DTYPE_BF16 ? launch_extend_bf16_q8(a, t, s) : launch_extend_f16_q8(a, t, s);
        else e = c.dtype == CONVT_DTYPE_BF16 ? launch_extend_bf16(a, t, s) : launch_extend_f16(a, t, s);
    } else {
        e = launch_extend_direct(a, c.dtype, c.quantised, s);
    }
    if (e == hipSuccess && a.chunks > 1) e = launch_extend_join(a, c.dtype, s);
    return device_status(e);
}

}  // namespace

extern "C" {

convt_status convt_cache_append(const convt_append_problem *problem, const void *q, const void *k, const void *v,
                                const int64_t *slots, const int64_t *positions, const float *inv_freq, void *k_cache,
                                void *v_cache, float *k_scale, float *v_scale, void *q_out, void *stream) {
    if (!problem) return CONVT_ERR_INVALID_ARGUMENT;
    const convt_append_problem &p = *problem;
    const convt_cache_desc &c = p.cache;
    const convt_status st = check_cache(c);
    if (st != CONVT_OK) return st;
    if (p.heads < 0 || p.reserved != 0 || !flag(p.interleaved)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.rotary_dim < 0 || p.rotary_dim > c.head_dim || p.rotary_dim % 2 != 0) return CONVT_ERR_INVALID_ARGUMENT;
    const int64_t per_token = (int64_t)p.heads + 2 * (int64_t)c.kv_heads;
    if (p.rows.tokens < 0 || p.rows.tokens > kMaxIndex || per_token > kMaxIndex || p.rows.tokens * per_token > kMaxIndex)
        return CONVT_ERR_INVALID_ARGUMENT;
    // a block's rows, at most 4 tokens', are counted in 32 bits
    if (per_token > kMaxIndex / 8) return CONVT_ERR_UNSUPPORTED;
    if (!strides_ok(p.rows.k_stride, 2, 0) || !strides_ok(p.rows.v_stride, 2, 0)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.heads > 0 && (!strides_ok(p.q_stride, 2, 0) || !strides_ok(p.q_out_stride, 2))) return CONVT_ERR_INVALID_ARGUMENT;
    if (!cache_pointers_ok(c, k_cache, v_cache, k_scale, v_scale)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.heads == 0 && (q || q_out)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.rows.tokens == 0) return CONVT_OK;
    if (!k || !v || !slots || (p.rotary_dim > 0 && (!positions || !inv_freq))) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.heads > 0 && (!q || !q_out)) return CONVT_ERR_INVALID_ARGUMENT;
    AppendArgs a{};
    a.c.k = k;
    a.c.v = v;
    a.c.k_cache = k_cache;
    a.c.v_cache = v_cache;
    a.c.k_scale = k_scale;
    a.c.v_scale = v_scale;
    a.c.slots = slots;
    for (int i = 0; i < 2; ++i) {
        a.c.row_stride[0][i] = p.rows.k_stride[i];
        a.c.row_stride[1][i] = p.rows.v_stride[i];
        a.q_stride[0][i] = p.q_stride[i];
        a.q_stride[1][i] = p.q_out_stride[i];
    }
    for (int i = 0; i < 3; ++i) {
        a.c.cache_stride[0][i] = c.k_stride[i];
        a.c.cache_stride[1][i] = c.v_stride[i];
    }
    a.c.n_slots = c.n_pages * c.page_size;
    a.c.tokens = p.rows.tokens;
    a.c.kv_heads = c.kv_heads;
    a.c.page_size = c.page_size;
    a.c.head_dim = c.head_dim;
    a.c.div_page = divisor_of((uint32_t)c.page_size);
    a.q = q;
    a.q_out = q_out;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.heads = p.heads;
    a.half = p.rotary_dim / 2;
    a.interleaved = p.interleaved;
    a.div_rows = divisor_of((uint32_t)per_token);
    a.div_half = divisor_of((uint32_t)(a.half > 0 ? a.half : 1));
    // tokens of a block: many amortise the angles, few spread over the card. Measured, us, with 1, 2, 4, 8: 32 + 8 heads of 128,
    // e4m3: 512 tokens: 6.3, 7.8, 11.8, 20.4; 1531: 11.8, 11.9, 15.4, 21.2; 3000: 19.3, 18.5, 18.9, 26.4; 4096: 24.0, 22.2, 22.8, 27.2;
    // 16384: 93.5, 84.1, 83.0, 86.7. 8 + 2 heads of 64, bf16: 512: 3.9, 3.7, 4.2, 4.7; 3000: 9.9, 7.2, 5.6, 5.7; 4096: 12.2, 8.3,
    // 6.5, 6.0; 16384: 40.8, 24.8, 17.0, 13.3 (few heads would take 4 from some 1000 tokens on).
    a.block_tokens = p.rows.tokens >= 4096 ? 4 : 1;
    return device_status(launch_append(a, c.dtype, c.quantised, (hipStream_t)stream));
}

convt_status convt_window_query(const convt_window_problem *problem, convt_extend_info *info) {
    if (!info) return CONVT_ERR_INVALID_ARGUMENT;
    Shape shape;
    return window_check(problem, info, &shape);
}

convt_status convt_window_attend(const convt_window_problem *problem, const void *q, const void *k_cache, const void *v_cache,
                                 const float *k_scale, const float *v_scale, const int32_t *page_table, const int32_t *lengths,
                                 const int32_t *starts, void *out, float *lse, void *workspace, void *stream) {
    convt_extend_info info;
    Shape shape;
    const convt_status st = window_check(problem, &info, &shape);
    if (st != CONVT_OK) return st;
    const convt_window_problem &p = *problem;
    const convt_cache_desc &c = p.cache;
    if (!cache_pointers_ok(c, k_cache, v_cache, k_scale, v_scale)) return CONVT_ERR_INVALID_ARGUMENT;
    if (!p.ragged && starts) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.batch == 0 || p.tokens == 0) return CONVT_OK;
    if (!q || !out || !lengths || (p.ragged && !starts) || (p.table_width > 0 && !page_table)) return CONVT_ERR_INVALID_ARGUMENT;
    if (info.workspace_bytes > 0 && (!workspace || !aligned(workspace, 16))) return CONVT_ERR_INVALID_ARGUMENT;
    ExtendArgs a = common_args(c, info, p.tokens, p.heads, p.max_length, p.scale, q, k_cache, v_cache, k_scale, v_scale, page_table,
                               lengths, out, lse, workspace);
    for (int i = 0; i < 2; ++i) {
        a.q_stride[1 + i] = p.q_stride[i];
        a.out_stride[1 + i] = p.out_stride[i];
    }
    a.table_stride = p.table_stride;
    a.batch = p.batch;
    a.starts = starts;
    // a window or first tokens beyond the longest stream are all of it
    a.window = p.window < p.max_length ? (int32_t)p.window : 0;
    a.sinks = p.sinks < p.max_length ? (int32_t)p.sinks : (int32_t)p.max_length;
    return launch(a, c, info, shape, (hipStream_t)stream);
}

convt_status convt_tree_query(const convt_tree_problem *problem, convt_extend_info *info) {
    if (!info) return CONVT_ERR_INVALID_ARGUMENT;
    Shape shape;
    return tree_check(problem, info, &shape);
}

convt_status convt_tree_attend(const convt_tree_problem *problem, const void *q, const void *k_cache, const void *v_cache,
                               const float *k_scale, const float *v_scale, const int32_t *page_table, const int32_t *lengths,
                               const uint64_t *tree, void *out, float *lse, void *workspace, void *stream) {
    convt_extend_info info;
    Shape shape;
    const convt_status st = tree_check(problem, &info, &shape);
    if (st != CONVT_OK) return st;
    const convt_tree_problem &p = *problem;
    const convt_cache_desc &c = p.cache;
    if (!cache_pointers_ok(c, k_cache, v_cache, k_scale, v_scale)) return CONVT_ERR_INVALID_ARGUMENT;
    if (p.batch == 0) return CONVT_OK;
    if (!q || !out || !lengths || !tree || (p.table_width > 0 && !page_table)) return CONVT_ERR_INVALID_ARGUMENT;
    if (!aligned(tree, 8)) return CONVT_ERR_INVALID_ARGUMENT;
    if (info.workspace_bytes > 0 && (!workspace || !aligned(workspace, 16))) return CONVT_ERR_INVALID_ARGUMENT;
    ExtendArgs a = common_args(c, info, (int64_t)p.batch * p.drafts, p.heads, p.max_length, p.scale, q, k_cache, v_cache, k_scale,
                               v_scale, page_table, lengths, out, lse, workspace);
    for (int i = 0; i < 3; ++i) {
        a.q_stride[i] = p.q_stride[i];
        a.out_stride[i] = p.out_stride[i];
    }
    a.tree_stride[0] = p.tree_stride[0];
    a.tree_stride[1] = p.tree_stride[1];
    a.table_stride = p.table_stride;
    a.batch = p.batch;
    a.drafts = p.drafts;
    a.div_drafts = divisor_of((uint32_t)p.drafts);
    a.tree = tree;
    return launch(a, c, info, shape, (hipStream_t)stream);
}

}  // extern "C"
