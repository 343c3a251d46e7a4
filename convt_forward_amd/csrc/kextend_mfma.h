// Attention of several new tokens per stream over the paged cache on the
// matrix cores: two-byte element types, caches of that type or of e4m3 codes.
// One kernel in three forms, for windows and for trees of drafts (a row: a
// token and a query head that shares the kv head; a wave has 32 of them):
//
//   many rows  tiles of 64 tokens go through LDS once for the rows of a block.
//         8 waves, 256 rows: the two waves of a SIMD take turns at products and
//         weights, with three buffers. For prompts and large trees, where the
//         matrix cores bound it.
//         4 waves, 128 rows, two blocks a CU that hide each other's beginnings and ends:
//         one barrier a tile, two buffers. For fewer rows.
//   few rows   4 waves with the same 32 rows; each takes every fourth tile of 32
//         tokens through its own part of LDS, without a barrier until the waves
//         are joined. Reading the cache bounds it.
//
//   scores  S^T = K Q^T by v_mfma_f32_32x32x16: A is 32 tokens x 16 dims of K, B
//           is Q, in registers. A lane then has one row (lane % 32) and 16 of a
//           sub-tile's 32 tokens, tokens 8 g + 4 (lane / 32) + i: a row's largest
//           score is over the lane's own values and one lane swap.
//   values  O^T += V^T P^T: B wants 8 tokens of the lane's row, which are 8
//           of the scores it holds, tokens 16 s + 4 (lane / 32) + i and those 8
//           further on; A wants the same tokens of one dim, which two transposing
//           LDS reads (4 tokens x 16 dims per 16 lanes each) give.
//   LDS     rows of K are spaced an odd number of 16 bytes modulo 256, those of
//           V 64 or 192: the reads then take all banks in turn.
//
// The running base of a row's exponents moves only when a score passes it by
// 2^8: rescaling O for every new maximum would cost as much as the
// exponentials. Weights over bfloat16 values carry 2^-8, so that none is above
// 1 and their products with the largest values stay finite.
//
// Roundings: Q and K enter as stored (e4m3 codes are exact in bf16 and f16;
// their scales multiply the float32 scores). Weights meet V
//   as float16 where V is float16 or e4m3 (its codes are exact there), 2^-11 of
//   their value. They carry a factor 2^7, so that those down to 2^-21 of
//   the base keep their 11 bits and smaller ones are off by at most 2^-32
//   of it. With e4m3 the logarithm of the value's scale is added to the score: the weight
//   is p times the scale, in float16's range whatever the scales are. The sum of p is that of the
//   weights times 1 / scale, which float32 holds for scales within 2^-40 .. 2^30. Values of smaller ones (rows of
//   zeros have 2^-126) are left out of it; a pass over the tiles that hold them adds their p at the end,
//   from the scores alone. Larger ones, or what is no number, make the sum NaN, and the pass forms it from all tiles.
//   A weight below 2^-60 of the row's largest may be lost where waves or parts are joined.
//   as the sum of two bfloat16 values (2^-16) in the form for few rows over
//   bfloat16, where the second product costs nothing beside the loads, and as one
//   (2^-8) in the forms for many, where it takes half as long again (a prompt of 8192
//   tokens 1.49 times as long, a large tree 1.43). Results then
//   are as far off as one more rounding of theirs: 0.0022 of their norm, 0.0016 without.
//
// Tokens that only some rows of a tile see: their scores become -infinity by
// a 64-bit mask per row, and infinite or NaN values among them (looked for
// in such tiles only) are left out of the product, which 0 times them would
// spoil. If there were any, a second pass over these tiles gives them to the
// rows that see them (inside the first one, its registers would have cost the
// others' prefetch).
//
// Measured (in a graph, 8 kv heads of 128, 4 query heads each): a prompt of 8192, window 4096, 16
// sinks, bf16: 449 us, 920 TFLOP/s. 64 drafts over 100 K and 131 K tokens, bf16: 343 us, 11 of them the
// join's, 2.9 TB/s and 730 TFLOP/s (327 back to back); 4 chunks of 512 over 2100 to 8000, e4m3: 233 us with the join. 64
// streams in a window of 4096, e4m3: 109 us, 4.7 TB/s (102 back to back). The pass for value scales far from 1: rows of
// zeros at the first token take 64 streams of 4096 from 118 to 130 us, a prompt of 4096 from 191 to 225; one
// scale of 2^31 there to 161 and 339. Tried and slower: 4 waves in the 8 waves'
// order of phases (1.08 times as long for the prompt), wave priorities around the products (1.01), two tiles on
// their way in registers (1.13). For the pass: in the loop, behind the weights (chunks 281 us, 250 without it) or before them
// (291), with a base of l's own in all tiles (278).
#pragma once

#include "extend.h"
#include "kdecode.h"
#include "kextend.h"

namespace convt {

namespace {

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// The other half-wave's value of the same row.
__device__ __forceinline__ float half_max(float v) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float half_sum(float v) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// 4 tokens of the lane's dim: 16 lanes give the addresses of 4 tokens x 16
// dims (4 dims each) and lane i of them gets dim i.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 read_transposed(const char *p) {
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p);
    return __builtin_bit_cast(u32x2, v);
}

// The n lowest of 64 bits.
__device__ __forceinline__ uint64_t low_bits(int n) {
    return n <= 0 ? 0 : n >= 64 ? ~(uint64_t)0 : ((uint64_t)1 << n) - 1;
}

// A word of two values with infinities and NaN replaced by 0; INF the bits of infinity.
template <uint32_t INF> __device__ __forceinline__ uint32_t word_finite(uint32_t w) {
    const uint32_t lo = (w & INF) == INF ? 0 : w & 0xffffu, hi = (w & (INF << 16)) == INF << 16 ? 0 : w & 0xffff0000u;
    return lo | hi;
}
// Four e4m3 codes with NaN, 0x7f of either sign, replaced by 0.
__device__ __forceinline__ uint32_t codes_finite(uint32_t w) {
    uint32_t r = 0;
    for (int i = 0; i < 4; ++i) r |= (w >> (8 * i) & 0x7f) == 0x7f ? 0 : w & 0xffu << (8 * i);
    return r;
}
// 1 (ONE its bits) where a value is of the kind: 0 infinity, 1 -infinity, 2 NaN.
template <uint32_t INF, uint32_t ONE> __device__ __forceinline__ uint32_t word_kind(uint32_t w, int kind) {
    uint32_t r = 0;
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = w >> (16 * i) & 0xffffu;
        const bool is = kind == 0 ? x == INF : kind == 1 ? x == (INF | 0x8000u) : (x & 0x7fffu) > INF;
        r |= is ? ONE << (16 * i) : 0;
    }
    return r;
}

constexpr int next_pow2(int n) { return n <= 1 ? 1 : 2 * next_pow2((n + 1) / 2); }

// The tiles that a part of the axis should have: all streams' tiles shared among the blocks that the card
// holds (tl.slots), so that ragged streams, whose lengths only the device knows, give it as
// many blocks as equal ones; tl.least at least. Unequal parts do not come out even on all
// shader engines, and one block too many takes as long as all: they get 0.85 of the
// card. Where the rows alone nearly fill it (0.6 of it), unequal streams are cut into smaller parts (1.7 times as many), so that the
// long ones end with the others. All blocks form the same number. 8 / 32 kv heads of 128, us:
//   0.6, 0.7, 0.85, 1 of the card: 16 trees of 25 drafts over 1 .. 4096 tokens, e4m3: 67, 60, 54, 68; 32 of 8 over
//   1 .. 8192, e4m3: 89, 83, 74, 76; 5 of 40 over 500 .. 20000, 64 dims: 77, 74, 76, 87; but 8 of 16 over 1 .. 16384, bf16:
//   83, 70, 98, 90, and 8 single tokens of 1 .. 32768, e4m3: 80, 69, 90, 85.
//   1, 1.35, 1.7, 2.2 times as many: 4 chunks of 512 over 2100 .. 8000, e4m3: 255, 257, 252, 276; 6 of 300 over 300 .. 12000,
//   e4m3: 310, 321, 275, 291; 8 of 256 over 256 .. 16384, bf16: 340, 328, 319, 318; but 16 of 128 over 128 .. 4096: 114, 120, 121, 121.
//   The border of nearly full at 0, 0.3, 0.6, 0.9: the 16 trees: 65, 54, 53, 53; the 4 chunks: 252, 252, 252, 318.
//   Unequal is a longest stream 1.05 times the mean: 4 equal trees of 64 over 16384: 103, taken as unequal 112; 16 trees
//   of 25 taken as equal: 67.
template <int KT> __device__ __forceinline__ float part_tiles(const ExtendArgs &a, const ExtendTiles &tl, int lane) {
    float sum = 0.0f, count = 0.0f, most = 0.0f;  // of the tiles that the last rows of each stream see, for each of its tiles of rows
    for (int b = lane; b < a.batch; b += 64) {
        int seen = cut_length(a, b), rows = tl.stream_tiles;
        if (a.window > 0 && seen - a.sinks > a.window) seen = a.window + a.sinks;
        if (rows == 0) {
            const int n = cut_start(a, b + 1) - cut_start(a, b);
            rows = n > 0 ? (n + tl.block_tokens - 1) / tl.block_tokens : 0;
        }
        const float tiles = (float)(seen / KT + 1);
        sum += (float)rows * tiles;
        count += (float)rows;
        most = fmaxf(most, tiles);
    }
    sum = wave_sum(sum);
    count = wave_sum(count);
    most = wave_max(most);
    const float each = (float)(tl.head_tiles * a.kv_heads), slots = (float)tl.slots;  // blocks of a tile of rows
    const float full = most * count < 1.05f * sum ? 1.0f : count * each < 0.6f * slots ? 0.85f : 1.7f;
    const float share = sum * each / (full * slots);
    return fmaxf(__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(share))), (float)(tl.least / KT));
}

// DP: head_dim rounded up to 64, 96, 128 or 256. WAVES: of a block, 8 only in the form for many rows.
template <typename E, bool Q8, int DP, bool KEYS, int WAVES, bool TREE>
__global__ __launch_bounds__(64 * WAVES, DP == 256 ? 1 : 2) void extend_mfma(ExtendArgs a, ExtendTiles tl) {
    typedef typename std::conditional<Q8, _Float16, E>::type EV;  // P and V
    typedef typename Vec8<E>::type E8;
    typedef typename Vec8<EV>::type EV8;
    constexpr bool SPLIT = KEYS && __is_same(EV, __bf16);
    constexpr float RAISE = __is_same(EV, __bf16) ? -8.0f : 7.0f;  // the weights carry 2^RAISE
    constexpr uint32_t INF = __is_same(EV, __bf16) ? 0x7f80u : 0x7c00u, ONE = __is_same(EV, __bf16) ? 0x3f80u : 0x3c00u;
    constexpr float SMALL = 0x1p-40f, LARGE = 0x1p30f;  // scales of e4m3 values that the sum of weights bears
    constexpr int KT = KEYS ? 32 : 64;           // tokens of a tile
    constexpr int NS = KT / 32, NG = KT / 16;
    constexpr int ROWS = KEYS ? 32 : 32 * WAVES; // of a block
    constexpr int GW = KEYS ? 2 : 1;             // groups of 16 tokens that a wave fills
    constexpr int SIDES = WAVES == 8 ? 1 : 2;    // K and V of them, or one of the two
    constexpr int CS = Q8 ? 1 : 2;               // bytes of a cache element
    constexpr int CHP = next_pow2(DP * CS / 16); // lanes along a token's row in the cache, 16 bytes each
    constexpr int RS = 64 / CHP;                 // rows they take at a time
    constexpr int NCH = 16 / RS;                 // pieces of a lane in a group
    constexpr int KSTR = DP * 2 + 16, VSTR = DP == 96 ? 192 : DP * 2 + 64;  // bytes between tokens in LDS
    constexpr int UNIT = KT * (KSTR + VSTR) + (Q8 ? 3 * KT * 4 : 0);
    constexpr int BUFFERS = WAVES == 8 ? 3 : 2;  // of tiles, in the form for many rows
    constexpr int NC = DP / 16, ND = DP / 32;
    __shared__ __attribute__((aligned(16))) char lds[(KEYS ? 4 : BUFFERS) * UNIT];
    __shared__ float m_lds[4][32], l_lds[4][32];
    __shared__ int there_lds[BUFFERS];  // whether a tile's groups have pages, a byte each

    const int lane = threadIdx.x % 64, r32 = lane % 32, h = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    // ---- the block's rows
    uint32_t at_block = blockIdx.x;
    auto digit = [&](const FastDiv &div, int of) {
        const uint32_t rest = fast_div(at_block, div);
        const int d = (int)(at_block - rest * (uint32_t)of);
        at_block = rest;
        return d;
    };
    const int kvh = digit(tl.div_kv, a.kv_heads);  // blocks of a kv head that follow each other go to one XCD's L2
    const int ht = digit(tl.div_head_tiles, tl.head_tiles);
    // the parts come last, so that the tiles that read the same tokens run together (the other way
    // round: 347 us against 240 for the chunks of 512 tokens)
    int tile = digit(tl.div_tiles, tl.tiles);
    const int chunk = (int)at_block;
    int b, tok0, end;  // the stream, the tile's first token, the end of the stream's tokens
    int len;           // the stream's cached tokens
    if (tl.stream_tiles > 0) {
        b = (int)fast_div((uint32_t)tile, tl.div_stream_tiles);
        const int in = tile - b * tl.stream_tiles;
        const int each = TREE ? a.drafts : 1;
        tok0 = b * each + in * tl.block_tokens;
        end = (b + 1) * each;
        len = cut_length(a, b);
    } else {
        // 64 streams at a time: the tiles up to each of them
        b = -1;
        tok0 = end = len = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 64) {
            int s0 = 0, s1 = 0, ln = 0;
            if (b0 + lane < a.batch) {
                s0 = cut_start(a, b0 + lane);
                s1 = cut_start(a, b0 + lane + 1);
                ln = cut_length(a, b0 + lane);
            }
            s1 = s1 < s0 ? s0 : s1;
            const int n = (int)fast_div((uint32_t)(s1 - s0 + tl.block_tokens - 1), tl.div_block_tokens);
            int sum = n;
            for (int d = 1; d < 64; d *= 2) {
                const int v = __shfl_up(sum, d);
                if (lane >= d) sum += v;
            }
            const uint64_t past = __ballot(sum > tile);
            if (past) {
                const int l = __ffsll((unsigned long long)past) - 1;
                b = b0 + l;
                // the last tiles of a stream see most and start first
                tok0 = __shfl(s0, l) + (__shfl(sum, l) - 1 - tile) * tl.block_tokens;
                end = __shfl(s1, l);
                len = __shfl(ln, l);
                break;
            }
            tile -= __shfl(sum, 63);
        }
        if (b < 0) return;  // the grid has room for the most tiles there can be
    }
    b = __builtin_amdgcn_readfirstlane(b);
    tok0 = __builtin_amdgcn_readfirstlane(tok0);
    end = __builtin_amdgcn_readfirstlane(end);
    len = __builtin_amdgcn_readfirstlane(len);
    const int nt = end - tok0 < tl.block_tokens ? end - tok0 : tl.block_tokens;
    const int hs = a.share - ht * ROWS < ROWS ? a.share - ht * ROWS : ROWS;  // heads of the tile
    const int nrows = nt * hs;
    const int row = KEYS ? r32 : wave * 32 + r32;
    const int real_row = row < nrows ? row : nrows - 1;  // rows past the last compute as it does and are not stored
    // quotients of numbers up to 256: half a step off a whole one, the reciprocal's rounding does not matter
    const float per_head = __builtin_amdgcn_rcpf((float)hs);
    auto of_head = [&](int r) { return (int)(((float)r + 0.5f) * per_head); };
    const int rt = of_head(real_row);
    const int token = tok0 + rt;
    const int head = kvh * a.share + ht * ROWS + real_row - rt * hs;
    // tokens of the wave's rows
    const bool idle = !KEYS && wave * 32 >= nrows;
    const int last = KEYS || wave * 32 + 31 >= nrows ? nrows - 1 : wave * 32 + 31;
    const int rt0 = __builtin_amdgcn_readfirstlane(KEYS ? 0 : of_head(wave * 32)), rt1 = __builtin_amdgcn_readfirstlane(of_head(last));

    // ---- what they see
    const int pos0 = TREE ? 0 : len - (end - tok0);  // position of the tile's first token
    int hi, first_seen = 0, sink_tiles = 0, base0 = 0;  // the last token that any row sees; the first ones before the window
    if constexpr (TREE) {
        hi = (len + a.drafts < a.max_length ? len + a.drafts : a.max_length) - 1;
    } else {
        hi = pos0 + nt - 1;
        const int lo = a.window > 0 && pos0 >= a.window ? pos0 - a.window + 1 : 0;
        first_seen = a.sinks < lo ? a.sinks : lo;
        sink_tiles = (first_seen + KT - 1) / KT;
        base0 = lo & ~15;
        if (base0 < sink_tiles * KT) base0 = sink_tiles * KT;
    }
    const int n_tiles = sink_tiles + (hi < base0 ? 0 : (hi - base0) / KT + 1);
    // This block's part of them: as many equal parts as the rows' share of the card's work is worth.
    int parts = 1;
    if (a.chunks > 1) {
        parts = (int)(n_tiles / part_tiles<KT>(a, tl, lane) + 0.4f);
        parts = parts < 1 ? 1 : parts > a.chunks ? a.chunks : parts;
        if (chunk >= parts) return;
    }
    const int per_part = (n_tiles + parts - 1) / parts;
    const int j0 = chunk * per_part;
    const int j1 = n_tiles - j0 < per_part ? n_tiles : j0 + per_part;
    const int64_t out_row = (int64_t)token * a.heads + head;
    const int64_t part = out_row * a.chunks + chunk;
    const int D = a.head_dim;
    auto tile_base = [&](int j) { return j < sink_tiles ? j * KT : base0 + (j - sink_tiles) * KT; };
    // The tiles that the rows of the tokens t0 .. t1 (of the block) all see whole: those before `first`,
    // of the first tokens, and from..to - 1.
    struct Whole {
        int first, from, to;
        __device__ bool has(int j) const { return j < first || (j >= from && j < to); }
    };
    auto whole_tiles = [&](int t0, int t1) {
        Whole w{0, 0, 0};
        if constexpr (TREE) {
            w.to = (len < hi + 1 ? len : hi + 1) / KT;
        } else {
            const int to = pos0 + t0 + 1 - base0, from = a.window > 0 ? pos0 + t1 - a.window + 1 - base0 : 0;
            w.first = first_seen / KT;
            w.from = sink_tiles + (from > 0 ? (from + KT - 1) / KT : 0);
            w.to = sink_tiles + (to > 0 ? to / KT : 0);
        }
        return w;
    };
    const Whole whole = whole_tiles(rt0, rt1), block_whole = KEYS ? whole : whole_tiles(0, nt - 1);
    const uint64_t *bits = nullptr;
    if constexpr (TREE) bits = a.tree + b * a.tree_stride[0] + (token - b * a.drafts) * a.tree_stride[1];
    // the tokens of a tile that the lane's row sees, `ok` the groups of 16 whose page is there
    auto seen_bits = [&](int base, uint32_t ok) {
        uint64_t seen;
        if constexpr (TREE) {
            seen = low_bits(len - base);
            const int d0 = base - len;  // the draft at the tile's first token
            const int words = (a.drafts + 63) / 64;
            if (d0 < 0) {
                if (d0 > -64) seen |= bits[0] << -d0;
            } else {
                const int w = d0 >> 6, s = d0 & 63;
                if (w < words) seen |= bits[w] >> s;
                if (s > 0 && w + 1 < words) seen |= bits[w + 1] << (64 - s);
            }
            seen &= low_bits(hi + 1 - base);
        } else {
            const int pos = pos0 + rt;
            seen = low_bits(pos + 1 - base);
            if (a.window > 0) seen &= ~low_bits(pos - a.window + 1 - base) | low_bits(a.sinks - base);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g)
            if (!(ok >> g & 1)) seen &= ~((uint64_t)0xffff << (16 * g));
        return seen;
    };

    // ---- Q, the B operand of the score products; a negative scale turns its sign
    const float c = a.scale_log2e == 0.0f ? 1.0f : fabsf(a.scale_log2e);
    E8 q[NC];
    {
        const uint16_t *qp = (const uint16_t *)a.q + head * a.q_stride[2];
        if constexpr (TREE) qp += b * a.q_stride[0] + (token - b * a.drafts) * a.q_stride[1];
        else qp += token * a.q_stride[1];
        const uint32_t flip = a.scale_log2e < 0.0f ? 0x80008000u : 0, keep = a.scale_log2e == 0.0f ? 0 : ~0u;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            u32x4 w = {0, 0, 0, 0};
            if (i * 16 < D) w = *(const u32x4 *)(qp + i * 16 + h * 8);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = (w[k] ^ flip) & keep;
            q[i] = __builtin_bit_cast(E8, w);
        }
    }

    // ---- filling tiles: a wave takes whole groups of 16 tokens, which lie in one page; of
    // 8 waves the first 4 take K and the others V
    const int g0 = KEYS ? 0 : wave % 4;  // the wave's first group of a tile
    auto is_v = [&](int side) { return SIDES == 2 ? side == 1 : wave >= 4; };
    const int r0 = lane / CHP, col = lane % CHP;
    const bool active = col * (16 / CS) < D;
    const char *cells[SIDES];
    uint32_t page_step[SIDES], token_step[SIDES];  // elements between pages, bytes between tokens
    uint32_t at_lane[SIDES][NCH];                  // the lane's bytes in a group (less than 2^30 by the route's rule)
#pragma unroll
    for (int s = 0; s < SIDES; ++s) {
        cells[s] = is_v(s) ? (const char *)a.v_cache + kvh * a.v_stride[1] * CS : (const char *)a.k_cache + kvh * a.k_stride[1] * CS;
        page_step[s] = (uint32_t)(is_v(s) ? a.v_stride[0] : a.k_stride[0]);
        token_step[s] = (uint32_t)(is_v(s) ? a.v_stride[2] : a.k_stride[2]) * CS;
#pragma unroll
        for (int i = 0; i < NCH; ++i) at_lane[s][i] = (r0 + i * RS) * token_step[s] + (active ? col : 0) * 16;
    }
    const int32_t *table = a.page_table + b * a.table_stride;
    char *my_lds = KEYS ? lds + wave * UNIT : lds;
    if (D < DP) {
        // the dims of K past D, which meet zeros of Q, are zeros; no piece is stored there
        for (int i = threadIdx.x * 4; i < (int)sizeof(lds); i += 64 * WAVES * 4) *(uint32_t *)(lds + i) = 0;
        __syncthreads();
    }
    u32x4 raw[SIDES][GW][NCH];
    float scale_raw[SIDES] = {};
    int32_t entry[GW];
    int entry_off[GW];
    uint32_t there = 0;  // the groups of the tile in the registers whose page is there
    // The pages of a tile's groups. A group past the end takes the last one
    // there is; its tokens are masked by their index.
    auto look_up = [&](int j) {
        const int base = tile_base(j < j1 ? j : j1 - 1) + 16 * g0;
#pragma unroll
        for (int g = 0; g < GW; ++g) {
            int t = base + 16 * g;
            t = t < (hi & ~15) ? t : hi & ~15;
            const int pi = (int)fast_div((uint32_t)t, a.div_page);
            entry[g] = table[pi];
            entry_off[g] = t - pi * a.page_size;
        }
    };
    auto load_tile = [&]() {
        there = 0;
#pragma unroll
        for (int g = 0; g < GW; ++g) {
            const bool ok = entry[g] >= 0 && entry[g] < a.n_pages;
            const uint32_t page = ok ? entry[g] : 0, off = entry_off[g];
            there |= ok ? 1u << g : 0;
#pragma unroll
            for (int s = 0; s < SIDES; ++s) {
                // strides of less than 2^31 elements: 32-bit factors
                const char *p = cells[s] + ((uint64_t)page * page_step[s] * CS + (uint64_t)off * token_step[s]);
#pragma unroll
                for (int i = 0; i < NCH; ++i) raw[s][g][i] = *(const u32x4 *)(p + at_lane[s][i]);
                if constexpr (Q8) {
                    const uint64_t at = (uint64_t)page * (uint32_t)(a.kv_heads * a.page_size) + (uint32_t)(kvh * a.page_size + (int)off);
                    // lanes 16 g .. of the groups' tokens; the others read what they do not use
                    const float v = (is_v(s) ? a.v_scale : a.k_scale)[at + (uint32_t)(lane % 16)];
                    scale_raw[s] = GW == 1 || lane / 16 == g ? v : scale_raw[s];
                }
            }
        }
    };
    // Where some row of the block does not see some token of the tile in the registers (edge), values that no row
    // sees become 0, infinities and NaN too unless `keep`. Returns whether there were any.
    auto clean_tile = [&](int base, bool edge, bool keep) {
        bool bad = false;
        if (edge || there != (1u << GW) - 1) {
#pragma unroll
            for (int s = 0; s < SIDES; ++s) {
                if (!is_v(s)) continue;
#pragma unroll
                for (int g = 0; g < GW; ++g)
#pragma unroll
                    for (int i = 0; i < NCH; ++i) {
                        const bool seen = base + 16 * (g0 + g) + r0 + i * RS <= hi && (there >> g & 1);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t x = seen ? raw[s][g][i][k] : 0, f = Q8 ? codes_finite(x) : word_finite<INF>(x);
                            bad |= edge && f != x;
                            raw[s][g][i][k] = edge && !keep ? f : x;
                        }
                    }
            }
        }
        return bad;
    };
    uint32_t odd = 0;  // 1: a tile that not all rows see held infinities or NaN, 2: a value's scale was too small for the sum
    // the tile at `base` to LDS; scales of values that no row sees are 1: what lies behind a stream would else bring
    // the pass for scales far from it
    auto store_tile = [&](char *to, int base) {
#pragma unroll
        for (int s = 0; s < SIDES; ++s) {
            constexpr int PW = Q8 ? 2 : 1;  // 16-byte words of LDS for one of the cache
#pragma unroll
            for (int g = 0; g < GW; ++g)
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    u32x4 w[PW];
                    if constexpr (Q8) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t x = raw[s][g][i][k];
                            uint32_t lo, hi2;
                            if constexpr (__is_same(E, EV)) {
                                lo = e4m3_pair<E, false>(x);
                                hi2 = e4m3_pair<E, true>(x);
                            } else {
                                lo = is_v(s) ? e4m3_pair<EV, false>(x) : e4m3_pair<E, false>(x);
                                hi2 = is_v(s) ? e4m3_pair<EV, true>(x) : e4m3_pair<E, true>(x);
                            }
                            w[k / 2][k % 2 * 2] = lo;
                            w[k / 2][k % 2 * 2 + 1] = hi2;
                        }
                    } else {
                        w[0] = raw[s][g][i];
                    }
                    const int r = 16 * (g0 + g) + r0 + i * RS;
                    char *p = to + (is_v(s) ? KT * KSTR + r * VSTR : r * KSTR) + col * (16 * PW);
                    if (active)
#pragma unroll
                        for (int k = 0; k < PW; ++k) *(u32x4 *)(p + 16 * k) = w[k];
                }
            if constexpr (Q8) {
                if (lane < 16 * GW) {
                    float *sp = (float *)(to + KT * (KSTR + VSTR)) + 16 * g0 + lane;
                    if (is_v(s)) {
                        const bool seen = base + 16 * g0 + lane <= hi && (there >> (lane / 16 % GW) & 1);
                        const float v = !seen ? 1.0f : scale_raw[s] < 0x1p-126f ? 0x1p-126f : scale_raw[s];
                        odd |= v < SMALL ? 2 : 0;
                        // the instructions alone, a step off each: v is no denormal number
                        sp[KT] = __builtin_amdgcn_logf(v);
                        sp[2 * KT] = v < SMALL ? 0.0f : v <= LARGE ? __builtin_amdgcn_rcpf(v) : __builtin_nanf("");
                    } else {
                        sp[0] = scale_raw[s] * c;
                    }
                }
            }
        }
    };

    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    float m = -INFINITY, l = 0.0f;  // the base of the weights (their largest is at most 2^(RAISE + 8)), their sum

    // byte offsets of the lane in a tile of K and of V
    const int k_at = r32 * KSTR + h * 16;
    const int v_at = KT * KSTR + (4 * h + lane % 16 / 4) * VSTR + (lane / 16 % 2 * 16 + lane % 4 * 4) * 2;

    f32x16 s[NS];                 // scores, then weights, of a tile
    u32x4 ph[NS * 2], pl[NS * 2]; // the weights as the B operand: their EV value, what it leaves
    auto scores = [&](const char *t) {
#pragma unroll
        for (int u = 0; u < NS; ++u) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const u32x4 w = *(const u32x4 *)(t + k_at + u * 32 * KSTR + i * 32);
                s[u] = mfma32(__builtin_bit_cast(E8, w), q[i], s[u]);
            }
        }
    };
    // The scores of what the row does not see become -infinity, by integers: as comparisons that two places of the kernel
    // make, each would keep a pair of scalar registers.
    auto mask = [&](int j, uint32_t ok) {
        const uint64_t seen = seen_bits(tile_base(j), ok) >> (4 * h);
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)(uint32_t)(seen >> (32 * u)), 8 * (i / 4) + i % 4, 1);
                s[u][i] = __uint_as_float((__float_as_uint(s[u][i]) & keep) | (0xff800000u & ~keep));
            }
    };
    auto weights = [&](const char *t, int j, uint32_t ok) {
        const float *sc = (const float *)(t + KT * (KSTR + VSTR)) + 4 * h;
        if constexpr (Q8) {
#pragma unroll
            for (int u = 0; u < NS; ++u)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 k = *(const f32x4 *)(sc + u * 32 + g * 8), v = *(const f32x4 *)(sc + KT + u * 32 + g * 8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[u][g * 4 + i] = __builtin_fmaf(s[u][g * 4 + i], k[i], v[i]);
                }
        }
        if (ok != (1u << NG) - 1 || !whole.has(j)) mask(j, ok);
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
        top = half_max(top);
        if constexpr (!Q8) top *= c;
        if (__any(top > m + (RAISE + 8.0f))) {
            const float up = fmaxf(m, top - RAISE);
            const float alpha = up == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - up);
            l *= alpha;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] *= alpha;
            m = up;
        }
        // scores of -infinity alone so far: any finite base
        const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[u][i] = __builtin_amdgcn_exp2f(Q8 ? s[u][i] - from : __builtin_fmaf(s[u][i], c, -from));
        if constexpr (Q8) {
#pragma unroll
            for (int u = 0; u < NS; ++u)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 v = *(const f32x4 *)(sc + 2 * KT + u * 32 + g * 8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) l = __builtin_fmaf(s[u][g * 4 + i], v[i], l);
                }
        } else {
#pragma unroll
            for (int u = 0; u < NS; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) l += s[u][i];
        }
#pragma unroll
        for (int k = 0; k < NS * 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = s[k / 2][k % 2 * 8 + 2 * i], y = s[k / 2][k % 2 * 8 + 2 * i + 1];
                ph[k][i] = pack_half2<EV>(x, y);
                if constexpr (SPLIT)
                    pl[k][i] = pack_half2<EV>(x - __uint_as_float(ph[k][i] << 16), y - __uint_as_float(ph[k][i] & 0xffff0000u));
            }
    };
    auto v_word = [&](const char *t, int k, int d) {  // 8 tokens of step k of 16, a dim of tile d
        const char *p = t + v_at + 16 * k * VSTR + d * 64;
        const u32x2 x = read_transposed(p), y = read_transposed(p + 8 * VSTR);
        return u32x4{x[0], x[1], y[0], y[1]};
    };
    auto values = [&](const char *t) {
#pragma unroll
        for (int k = 0; k < NS * 2; ++k)
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                u32x4 w = v_word(t, k, d);
                o[d] = mfma32(__builtin_bit_cast(EV8, w), __builtin_bit_cast(EV8, ph[k]), o[d]);
                if constexpr (SPLIT) {
                    // the low part may be 0 or negative: an infinite value takes part in the first product only
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = finite_bf16(w[i]);
                    o[d] = mfma32(__builtin_bit_cast(EV8, w), __builtin_bit_cast(EV8, pl[k]), o[d]);
                }
            }
    };
    // The order of a phase's LDS reads and products: operands are read two groups of 4 ahead of their
    // products. Left alone the compiler reads two operands and waits for both: 1570
    // cycles for the products of a tile of 64 tokens and 128 dims, 1290 so.
    constexpr int GV = NS * 2 * ND / 4, GK = NS * NC / 4;
    constexpr int READ = 0x100, PRODUCT = 0x8;  // LDS reads (two for an operand of V) and matrix instructions
    auto order_scores = [&]() {
        __builtin_amdgcn_sched_group_barrier(READ, GK > 1 ? 8 : 4, 0);
#pragma unroll
        for (int i = 2; i < GK; ++i) {
            __builtin_amdgcn_sched_group_barrier(PRODUCT, 4, 0);
            __builtin_amdgcn_sched_group_barrier(READ, 4, 0);
        }
        __builtin_amdgcn_sched_group_barrier(PRODUCT, GK > 1 ? 8 : 4, 0);
    };
    auto order_values = [&]() {
        __builtin_amdgcn_sched_group_barrier(READ, GV > 1 ? 16 : 8, 0);
#pragma unroll
        for (int i = 2; i < GV; ++i) {
            __builtin_amdgcn_sched_group_barrier(PRODUCT, 4, 0);
            __builtin_amdgcn_sched_group_barrier(READ, 8, 0);
        }
        __builtin_amdgcn_sched_group_barrier(PRODUCT, GV > 1 ? 8 : 4, 0);
    };
    // The same with the order written out, where hints do not hold (they do until code elsewhere takes another register): an
    // operand is read RING products ahead of its own, STEP at a time. The 8 waves' phase multiplies the values of a tile,
    // whose first operands are there, and the scores of the next one; the 4 waves' two phases over e4m3 each do one
    // of them. With a wait for each operand a prompt of 4096 over e4m3 takes 219 us, 190 so (as with 4 to 12 ahead; 203 where nothing
    // else may move between them, though a long tree over bf16 takes 328 then, 343 so); 16 trees of 25 drafts 61, 57 so
    // (60 with 8 ahead, whose registers spill).
    constexpr int PASS = 0x2 | 0x4 | 0x20;  // what may move between them: other arithmetic, global loads
    constexpr int RING = WAVES == 8 ? 8 : 4, STEP = RING / 2, NV = NS * 2 * ND, NP = NV + NS * NC;
    u32x4 ring[RING];
    auto operand = [&](const char *t, const char *next, int f) {
        const int c = f - NV;
        return f < NV ? v_word(t, f / ND, f % ND) : *(const u32x4 *)(next + k_at + c / NC * 32 * KSTR + c % NC * 32);
    };
    auto read_ahead = [&](const char *t, int from) {
#pragma unroll
        for (int f = from; f < from + RING; ++f) ring[f % RING] = operand(t, t, f);
    };
    auto products = [&](const char *t, const char *next, int from, int to) {
        if (to > NV)
#pragma unroll
            for (int u = 0; u < NS; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
        for (int f0 = from; f0 < to; f0 += STEP) {
            __builtin_amdgcn_sched_barrier(PASS);
#pragma unroll
            for (int f = f0; f < f0 + STEP; ++f) {
                const int c = f - NV;
                if (f < NV) o[f % ND] = mfma32(__builtin_bit_cast(EV8, ring[f % RING]), __builtin_bit_cast(EV8, ph[f / ND]), o[f % ND]);
                else s[c / NC] = mfma32(__builtin_bit_cast(E8, ring[f % RING]), q[c % NC], s[c / NC]);
            }
#pragma unroll
            for (int f = f0 + RING; f < f0 + RING + STEP && f < to; ++f) ring[f % RING] = operand(t, next, f);
        }
        __builtin_amdgcn_sched_barrier(PASS);
    };
    // Infinities and NaN of a tile that not all rows see: for each kind, whether the row sees one in the dim.
    auto add_kinds = [&](const char *t, int base) {
        const uint64_t seen = seen_bits(base, ~0u) >> (4 * h);
#pragma unroll 1
        for (int kind = 0; kind < 3; ++kind) {
            const float add = kind == 0 ? INFINITY : kind == 1 ? -INFINITY : __builtin_nanf("");
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                f32x16 any;
#pragma unroll
                for (int i = 0; i < 16; ++i) any[i] = 0.0f;
#pragma unroll
                for (int k = 0; k < NS * 2; ++k) {
                    u32x4 w = v_word(t, k, d), sees;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[i] = word_kind<INF, ONE>(w[i], kind);
                        const int at = 16 * k + 8 * (i / 2) + 2 * (i % 2);
                        sees[i] = (seen >> at & 1 ? ONE : 0) | (seen >> (at + 1) & 1 ? ONE << 16 : 0);
                    }
                    any = mfma32(__builtin_bit_cast(EV8, w), __builtin_bit_cast(EV8, sees), any);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] = any[i] > 0.0f ? o[d][i] + add : o[d][i];
            }
        }
    };

    // The pass for scales that the sum of weights does not bear: l to a base of its own, a whole number, so that it
    // moves by powers of two. `all`: from the beginning.
    float ml = 0.0f;
    auto move_sum = [&](float to) {
        const float up = fmaxf(ml, floorf(to));
        l *= up == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(ml - up);
        ml = up;
    };
    auto begin_plain = [&](bool all) {
        ml = all ? -INFINITY : m;
        l = all ? 0.0f : l;
        move_sum(all ? -INFINITY : m + 1.0f);
    };
    // whether the lane's token of tile j (after look_up) has a value of a small scale
    auto has_low = [&](int j) {
        const int g = lane / 16 % GW, t = tile_base(j) + 16 * g0 + lane;
        int32_t page = entry[0];
        int off = entry_off[0];
        if (GW == 2 && g == 1) {
            page = entry[GW - 1];
            off = entry_off[GW - 1];
        }
        if (lane >= 16 * GW || t > hi || page < 0 || page >= a.n_pages) return false;
        return a.v_scale[((int64_t)page * a.kv_heads + kvh) * a.page_size + off + lane % 16] < SMALL;
    };
    // adds the p of a tile's tokens, or of those with a small scale
    auto add_plain = [&](const char *t, int j, uint32_t ok, bool all) {
        scores(t);
        const float *sc = (const float *)(t + KT * (KSTR + VSTR)) + 4 * h;
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 k = *(const f32x4 *)(sc + u * 32 + g * 8), r = *(const f32x4 *)(sc + 2 * KT + u * 32 + g * 8);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[u][g * 4 + i] = all || r[i] == 0.0f ? s[u][g * 4 + i] * k[i] : -INFINITY;
            }
        mask(j, ok);
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
        move_sum(half_max(top));
        const float from = ml == -INFINITY ? 0.0f : ml;
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) l += __builtin_amdgcn_exp2f(s[u][i] - from);
    };
    // O to the base of l, and l to 0.5 .. 1: in two steps, as 2^(m - base) may pass float32's range
    auto end_plain = [&]() {
        const float both = half_sum(l);
        const int e = __builtin_amdgcn_frexp_expf(both);
        const float half = both == 0.0f ? 1.0f : __builtin_amdgcn_exp2f(0.5f * (m - ml - (float)e));
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = o[d][i] * half * half;
        m = both == 0.0f ? -INFINITY : ml + (float)e;
        l = h == 0 ? __builtin_amdgcn_frexp_mantf(both) : 0.0f;
    };

    if constexpr (KEYS) {
        // the tile is the wave's own: its stores are done before its reads, and those before the next stores
        auto own_order = [&]() {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };
        int j = j0 + wave;
        if (j < j1) {
            look_up(j);
            load_tile();
            look_up(j + 4);
        }
        for (; j < j1; j += 4) {
            const uint32_t ok = there;
            odd |= clean_tile(tile_base(j), !whole.has(j), false);
            store_tile(my_lds, tile_base(j));
            own_order();
            load_tile();  // the wave's next one; past the end the last one, which is not used
            look_up(j + 8);
            scores(my_lds);
            order_scores();
            weights(my_lds, j, ok);
            values(my_lds);
            order_values();
            own_order();
        }
        if (__any(odd & 1))
            for (j = j0 + wave; j < j1; j += 4) {
                if (whole.has(j)) continue;
                look_up(j);
                load_tile();
                clean_tile(tile_base(j), true, true);
                store_tile(my_lds, tile_base(j));
                own_order();
                add_kinds(my_lds, tile_base(j));
                own_order();
            }
        if constexpr (Q8)
            if (__any((odd & 2) || l != l)) {
                const bool all = __any(l != l);
                begin_plain(all);
                for (j = j0 + wave; j < j1; j += 4) {
                    look_up(j);
                    if (!all && !__any(has_low(j))) continue;
                    load_tile();
                    store_tile(my_lds, tile_base(j));
                    own_order();
                    add_plain(my_lds, j, there, all);
                    own_order();
                }
                end_plain();
            }
    } else if (j0 < j1) {
        // Tile j, which is in the registers (past the end the last one again).
        auto clean = [&](int j, bool keep) {
            j = j < j1 ? j : j1 - 1;
            odd |= clean_tile(tile_base(j), !block_whole.has(j), keep);
        };
        auto store = [&](int buffer, int j, bool flags) {
            store_tile(lds + buffer * UNIT, tile_base(j < j1 ? j : j1 - 1));
            if (flags && lane == 0 && wave < 4) ((uint8_t *)&there_lds[buffer])[wave] = (uint8_t)there;
        };
        look_up(j0);
        load_tile();
        look_up(j0 + 1);
        // whether any page of the block's tiles is outside the cache: only then tiles have flags
        bool outside = false;
        {
            const int t0 = tile_base(j0 < sink_tiles ? sink_tiles : j0), t1 = tile_base(j1 - 1) + KT - 1;
            const int last_page = (int)fast_div((uint32_t)(t1 < hi ? t1 : hi), a.div_page);
            for (int p = (int)fast_div((uint32_t)t0, a.div_page) + (int)threadIdx.x; p <= last_page; p += 64 * WAVES)
                outside |= table[p] < 0 || table[p] >= a.n_pages;
            for (int j = j0; j < sink_tiles; ++j)
                for (int g = (int)threadIdx.x; g < NG; g += 64 * WAVES) {
                    const int p = (int)fast_div((uint32_t)(j * KT + 16 * g < hi ? j * KT + 16 * g : hi), a.div_page);
                    outside |= table[p] < 0 || table[p] >= a.n_pages;
                }
        }
        clean(j0, false);
        store(0, j0, true);
        load_tile();
        look_up(j0 + 2);
        const bool flags = __syncthreads_or(outside);
        // the groups of a tile that have pages, from a byte for each
        auto ok_of = [&](int buffer) {
            uint32_t ok = (1u << NG) - 1;
            if (flags) ok = ((uint32_t)__builtin_amdgcn_readfirstlane(there_lds[buffer]) * 0x01020408u) >> 24;
            return ok;
        };
        int at = 0;  // the buffer of tile j
        if constexpr (WAVES == 4) {
            for (int j = j0; j < j1; ++j, at ^= 1) {
                const char *t = lds + at * UNIT;
                if (!idle) {
                    if constexpr (Q8) {
                        read_ahead(t, NV);
                        products(t, t, NV, NP);
                    } else {
                        scores(t);
                        order_scores();
                    }
                }
                // behind the products
                clean(j + 1, false);
                store(at ^ 1, j + 1, flags);
                load_tile();
                look_up(j + 3);
                if (!idle) {
                    weights(t, j, ok_of(at));
                    if constexpr (Q8) {
                        read_ahead(t, 0);
                        products(t, t, 0, NV);
                    } else {
                        values(t);
                        order_values();
                    }
                }
                __syncthreads();
            }
        } else {
            // The two waves of a SIMD take turns: while one multiplies (the values of tile j, then the
            // scores of tile j + 1) the other forms weights. Phases, counted from the first waves'
            // scores of tile j0, with n = j - j0: these form the weights of tile j in phase 2 n + 1 and
            // multiply in 2 n + 2, the others one phase later. The phase that multiplies
            // for tile j also fills tile j + 2's buffer, of three: tile j - 1 was in it, whose values
            // the others read last in phase 2 n + 1. Tile j + 2 is first read in phase 2 n + 4.
            auto next = [&](int b, int by) { return b + by < 3 ? b + by : b + by - 3; };
            const bool second = wave >= 4;
            if (second) __syncthreads();
            if (idle) {
                clean(j0 + 1, false);
                store(1, j0 + 1, flags);
                load_tile();
                __syncthreads();
                for (int j = j0; j < j1; ++j) {
                    look_up(j + 3);
                    clean(j + 2, false);
                    __syncthreads();
                    store(next(at, 2), j + 2, flags);
                    load_tile();
                    __syncthreads();
                    at = next(at, 1);
                }
            } else {
                scores(lds);
                clean(j0 + 1, false);
                store(1, j0 + 1, flags);
                load_tile();
                __syncthreads();
                for (int j = j0; j < j1; ++j) {
                    const char *t = lds + at * UNIT;
                    look_up(j + 3);
                    weights(t, j, ok_of(at));
                    // in this phase: the compiler would move them to where they are used, behind the barrier
#pragma unroll
                    for (int k = 0; k < NS * 2; ++k) asm volatile("" : "+v"(ph[k]));
                    asm volatile("" : "+v"(l));
                    read_ahead(t, 0);
                    clean(j + 2, false);
                    __syncthreads();
                    store(next(at, 2), j + 2, flags);
                    load_tile();  // of j + 3
                    products(t, lds + next(at, 1) * UNIT, 0, NP);  // past the end of the last tile again, which is not used
                    __syncthreads();
                    at = next(at, 1);
                }
            }
            if (!second) __syncthreads();
        }
        if (__syncthreads_or(odd & 1))
            for (int j = j0; j < j1; ++j) {
                if (block_whole.has(j)) continue;
                look_up(j);
                load_tile();
                clean(j, true);
                store(0, j, false);
                __syncthreads();
                if (!idle) add_kinds(lds, tile_base(j));
                __syncthreads();
            }
        if constexpr (Q8)
            if (__syncthreads_or((odd & 2) || l != l)) {
                const bool all = __syncthreads_or(l != l);
                begin_plain(all);
                for (int j = j0; j < j1; ++j) {
                    look_up(j);
                    if (!all && !__syncthreads_or(has_low(j))) continue;
                    load_tile();
                    store(0, j, flags);
                    __syncthreads();
                    if (!idle) add_plain(lds, j, ok_of(0), all);
                    __syncthreads();
                }
                end_plain();
            }
    }

    // ---- results: the lane has dims 32 d + 8 g + 4 h + i of its row
    auto store_row = [&](float mm, float ll, auto value) {
        // value(d, g): 4 dims of the row
        const bool whole = parts == 1;
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        uint16_t *op = nullptr;
        if (whole) {
            op = (uint16_t *)a.out + head * a.out_stride[2];
            if constexpr (TREE) op += b * a.out_stride[0] + (token - b * a.drafts) * a.out_stride[1];
            else op += token * a.out_stride[1];
        }
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int at = 32 * d + 8 * g + 4 * h;
                if (at >= D) continue;
                const f32x4 v = value(d, g);
                if (whole) {
                    typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
                    f32x4 x;
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = ll == 0.0f ? 0.0f : v[i] * inv;
                    *(u32x2_a2 *)(op + at) = u32x2{pack_half2<E>(x[0], x[1]), pack_half2<E>(x[2], x[3])};
                } else {
                    *(f32x4 *)(a.part_o + part * D + at) = v;
                }
            }
        if (h == 0) {
            if (!whole) {
                a.part_ml[part * 2] = mm;
                a.part_ml[part * 2 + 1] = ll;
            } else if (a.lse) {
                a.lse[out_row] = (mm + log2f(ll)) * 0.69314718055994531f;
            }
            // for the join: how many parts there are, none if the row is done
            if (a.chunks > 1 && chunk == 0) a.part_count[out_row] = whole ? 0 : parts;
        }
    };
    l = half_sum(l);
    if constexpr (!KEYS) {
        if (row < nrows)
            store_row(m, l, [&](int d, int g) { return f32x4{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]}; });
    } else {
        // Join the waves: each brings its O to the common base and leaves it in LDS, then takes a quarter of the rows' dims.
        if (h == 0) {
            m_lds[wave][r32] = m;
            l_lds[wave][r32] = l;
        }
        __syncthreads();  // every wave is done with its tiles
        float mm = -INFINITY, ll = 0.0f;
        for (int w = 0; w < 4; ++w) mm = fmaxf(mm, m_lds[w][r32]);
        const float from = mm == -INFINITY ? 0.0f : mm;
        for (int w = 0; w < 4; ++w) ll += l_lds[w][r32] * __builtin_amdgcn_exp2f(m_lds[w][r32] - from);
        const float f = __builtin_amdgcn_exp2f(m - from);
        float *ol = (float *)lds;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = o[d][4 * g + i] * f;
                *(f32x4 *)(ol + ((wave * ND + d) * 4 + g) * 256 + lane * 4) = v;
            }
        __syncthreads();
        if (wave == 0 && row < nrows)
            store_row(mm, ll, [&](int d, int g) {
                f32x4 v = *(const f32x4 *)(ol + (d * 4 + g) * 256 + lane * 4);
                for (int w = 1; w < 4; ++w) v += *(const f32x4 *)(ol + ((w * ND + d) * 4 + g) * 256 + lane * 4);
                return v;
            });
    }
}

template <typename E, bool Q8, int DP, bool TREE> void run_form(const ExtendArgs &a, const ExtendTiles &t, hipStream_t s) {
    const unsigned grid = (unsigned)t.tiles * (unsigned)t.head_tiles * (unsigned)a.kv_heads * (unsigned)a.chunks;
    if (t.form == ExtendForm::kKeys) extend_mfma<E, Q8, DP, true, 4, TREE><<<grid, 256, 0, s>>>(a, t);
    else if (t.form == ExtendForm::kRows128) extend_mfma<E, Q8, DP, false, 4, TREE><<<grid, 256, 0, s>>>(a, t);
    else if constexpr (DP <= 128) extend_mfma<E, Q8, DP, false, 8, TREE><<<grid, 512, 0, s>>>(a, t);
}

template <typename E, bool Q8, int DP> void run_extend(const ExtendArgs &a, const ExtendTiles &t, hipStream_t s) {
    if (a.tree) run_form<E, Q8, DP, true>(a, t, s);
    else run_form<E, Q8, DP, false>(a, t, s);
}

template <typename E, bool Q8> hipError_t run_dims(const ExtendArgs &a, const ExtendTiles &t, hipStream_t s) {
    if (a.head_dim <= 64) run_extend<E, Q8, 64>(a, t, s);
    else if (a.head_dim <= 96) run_extend<E, Q8, 96>(a, t, s);
    else if (a.head_dim <= 128) run_extend<E, Q8, 128>(a, t, s);
    else run_extend<E, Q8, 256>(a, t, s);
    return hipGetLastError();
}

}  // namespace

}  // namespace convt
