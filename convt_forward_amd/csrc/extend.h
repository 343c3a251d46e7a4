// Parameters and launchers of the kernels for several new tokens per stream
// (host side: checked in extend_api.cpp before any launch).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "convt_extend.h"
#include "decode.h"

namespace convt {

struct AppendArgs {
    CacheArgs c;                  // k and v, the cache, slots
    const void *q;
    void *q_out;
    const int64_t *positions;
    const float *inv_freq;
    int64_t q_stride[2][2];       // [q, q_out][token, head]
    int32_t heads, half;          // half = rotary_dim / 2
    int32_t interleaved, block_tokens;
    FastDiv div_rows, div_half;   // by heads + 2 kv_heads, by max(half, 1)
};
hipError_t launch_append(const AppendArgs &a, int dtype, int quantised, hipStream_t stream);

struct ExtendArgs {
    const void *q, *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *page_table, *lengths;
    const int32_t *starts;        // window: NULL for one token per stream
    const uint64_t *tree;         // tree: not NULL
    void *out;
    float *lse;
    // workspace: [tokens * heads][chunks][head_dim], [..][chunks][2], [..]: the row's parts,
    // 0 for a row that is done without them
    float *part_o, *part_ml;
    int32_t *part_count;
    int64_t q_stride[3], out_stride[3];  // batch (tree), token, head
    int64_t k_stride[3], v_stride[3];
    int64_t tree_stride[2];
    int64_t table_stride, n_pages;
    int32_t batch, tokens;        // tokens: rows of q; tree: batch * drafts
    int32_t drafts;               // tree: new tokens of a stream
    int32_t heads, kv_heads, share;  // share = heads / kv_heads
    int32_t head_dim, page_size, max_length;
    int32_t window, sinks;        // window 0: no limit
    int32_t chunks, chunk_tokens;  // parts at most; tokens of one in the direct kernel
    float scale_log2e;            // scale * log2(e): the softmax runs on powers of two
    FastDiv div_page, div_heads, div_drafts;
};
hipError_t launch_extend_direct(const ExtendArgs &a, int dtype, int quantised, hipStream_t stream);

// The forms of the matrix-core kernel (kextend_mfma.h): few rows, whose waves
// share the tokens, and 128 or 256 rows a block.
enum class ExtendForm : int32_t { kKeys, kRows128, kRows256 };

// How a launch's blocks of the matrix-core kernel map to the rows.
struct ExtendTiles {
    ExtendForm form;
    int32_t block_tokens;   // tokens of a tile of rows
    int32_t head_tiles;     // tiles of the query heads that share a kv head
    int32_t stream_tiles;   // tiles of a stream where all have the same number (trees, no starts), else 0
    int32_t tiles;          // of the grid
    int32_t slots;          // blocks that the card holds at once
    int32_t least;          // tokens that a part has at least
    FastDiv div_kv, div_head_tiles, div_tiles, div_stream_tiles, div_block_tokens;
};
hipError_t launch_extend_bf16(const ExtendArgs &a, const ExtendTiles &t, hipStream_t stream);
hipError_t launch_extend_f16(const ExtendArgs &a, const ExtendTiles &t, hipStream_t stream);
hipError_t launch_extend_bf16_q8(const ExtendArgs &a, const ExtendTiles &t, hipStream_t stream);
hipError_t launch_extend_f16_q8(const ExtendArgs &a, const ExtendTiles &t, hipStream_t stream);
hipError_t launch_extend_join(const ExtendArgs &a, int dtype, hipStream_t stream);

}  // namespace convt
