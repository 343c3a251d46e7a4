// Products of a few rows with 4-bit weights and group scales on the matrix
// cores (two-byte element types, groups of 32, 64 or 128).
//
// Reading the weights bounds it (HBM), and next to that unpacking them: at 8
// TB/s a CU receives 26 weights a clock and has 64 vector lanes, so a weight
// may cost about two lane operations. The byte 0000wwww is the e4m3 value
// w * 2^-9, below and above that type's normal range alike, so a shift and two
// ands make the bytes of 8 weights and four conversions (with the scale 2^9)
// the E values w, 7 operations in all, exactly. (Placing the bits into the
// mantissa of 16.0 takes 8, for 16 + w: 37 against 34 us for the case below.)
// The 8 that w is too large by is taken off as 8 sum x of the group: one more
// product, of x with a constant, whose result is where the group's sum
// starts. All products are exact in float32; the sums' roundings are those of
// terms up to 15 |x|, twice the 8 |x| of w - 8 itself. Where most w - 8 are small
// and x is of one sign the two sums are larger than what is left of them: the error
// stays 2^-24 of their size (weights of 0 alone, 4096 x in 0 .. 1: up to 1e-4
// where sum 8 |x| is 16600), which matters to a two-byte result only below
// 2^-12 of sum 8 |x|. e4m3 rows are widened to E, exactly, for
// the same products: those on 8-bit operands would take the weights' bytes
// as they are, but they line their terms up with fewer bits than float32
// has (off by up to 6e-6 of the terms' magnitudes at k = 128, where these stay
// below 6e-9).
// One product serves up to 16 rows of x, and a group's scale multiplies its
// finished sum, once for 4 results.
//
// v_mfma_f32_16x16x32: A is 16 rows of x, B 16 columns (n) of W, a lane 8
// consecutive k of one. Loads of W are 16 bytes of one n a lane, 32 k, so that
// the four lanes of an n hold 128 k; each product wants its 32 k from four
// lanes, 8 each, so the words are transposed among the four lanes (4 lane
// swaps for 4 words) and every group of 32 k or more stays in one product.
// (e4m3 x with groups of 128 takes the lanes' own 32 k of both instead.)
// Unpacking leaves the even k of a word before the odd ones, and x is brought
// to that order; the sum does not mind.
//
// Waves of a block share columns with different k (WK of them, joined through
// LDS at the end) or take other columns (WN).
//
// Measured: 16 e4m3 rows x 8192 x 32768 (134 MB of weights): 34 us, 4.1 TB/s; its
// weights' loads alone take 25, x (read by every block through the caches)
// most of the rest. One bf16 row: 31 us. One row x 4096 x 4096, 8.7 MB: 4.6
// us a call of a graph (5.4 in a kernel trace); an empty launch takes 2.5, a
// bare read of 8 MB 2.5 with its launch.
#include "decode.h"
#include "kdecode.h"

namespace convt {

namespace {

struct Q4Args {
    const void *x, *w, *scales;
    const float *x_scale;
    void *y;
    int64_t x_stride, y_stride;
    int32_t rows, n, k, groups;
    int32_t wk, wn;              // waves of a block over k, over columns
    int32_t each;                // stages of a wave
    int32_t scale_row;           // LDS: elements of a column's scales
    int32_t x_at, x_row;         // LDS with XL: byte offset of x, bytes of a row of it
};

constexpr int kMaxWaves = 8;  // of a block

// 8 weights, as they are, in the order (0, 2), (4, 6), (1, 3), (5, 7).
template <typename E> __device__ __forceinline__ typename Vec8<E>::type unpack(uint32_t w) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
    return __builtin_bit_cast(typename Vec8<E>::type, u32x4{e4m3_pair<E, false>(even, 512.0f), e4m3_pair<E, true>(even, 512.0f),
                                                           e4m3_pair<E, false>(odd, 512.0f), e4m3_pair<E, true>(odd, 512.0f)});
}

// 8 consecutive x in the same order.
template <typename E> __device__ __forceinline__ typename Vec8<E>::type order_x(u32x4 w) {
    return __builtin_bit_cast(typename Vec8<E>::type, u32x4{lo_pair(w[0], w[1]), lo_pair(w[2], w[3]),
                                                           hi_pair(w[0], w[1]), hi_pair(w[2], w[3])});
}
template <typename E> __device__ __forceinline__ typename Vec8<E>::type order_x(u32x2 w) {
    const uint32_t even = __builtin_amdgcn_perm(w[1], w[0], 0x06040200u), odd = __builtin_amdgcn_perm(w[1], w[0], 0x07050301u);
    return __builtin_bit_cast(typename Vec8<E>::type, u32x4{e4m3_pair<E, false>(even), e4m3_pair<E, true>(even),
                                                           e4m3_pair<E, false>(odd), e4m3_pair<E, true>(odd)});
}

// Word j of lane group g <-> word g of lane group j (groups of 16 lanes).
__device__ __forceinline__ u32x4 transpose_groups(u32x4 w) {
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

// NT: tiles of 16 columns a wave, MT: tiles of 16 rows of x, U: chunks of 128 k a
// stage, XL: x is held in LDS.
template <typename E, bool X8, int GS, int NT, int MT, int U, bool XL>
__global__ __launch_bounds__(64 * kMaxWaves) void q4_mfma(Q4Args a) {
    typedef typename Vec8<E>::type E8;
    constexpr int XS = X8 ? 1 : 2;
    // x of a chunk in 16-byte pieces of a lane: 8 k each for the products of 32 k, or, of
    // e4m3 rows, the lane's own 32 k, as W has them
    constexpr int NX = X8 ? 2 : 4, XLANE = X8 ? 32 : 8, XSTEP = X8 ? 16 : 32;
    // Where a product may mix the chunk's 32 k of each lane group (one group of
    // weights), e4m3 x and W stay in the lanes they were loaded into.
    constexpr bool STAY = X8 && GS == 128;
    constexpr int G = 128 / GS;  // groups of a chunk
    constexpr int GU = G * U;    // groups of a stage
    // The block's scales, a row of scale_row for each of its columns, and x with
    // XL; then the waves' sums.
    extern __shared__ f32x4 lds[];
    const int lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wk = wave % a.wk, wn = wave / a.wk;
    const int m0 = blockIdx.y * 16 * MT;
    const int tile0 = (blockIdx.x * a.wn + wn) * NT;  // first tile of 16 columns

    const char *wp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        // columns past the last read the last one and are not stored
        int64_t n = (int64_t)(tile0 + t) * 16 + r;
        n = n < a.n ? n : a.n - 1;
        wp[t] = (const char *)a.w + n * (a.k / 2) + g * 16;
    }
    const char *xp[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        // rows past the last read the last one: their results are not stored
        int m = m0 + mt * 16 + r;
        m = m < a.rows ? m : a.rows - 1;
        xp[mt] = (const char *)a.x + (m * a.x_stride + g * XLANE) * XS;
    }

    struct Stage {
        u32x4 w[U][NT];
        u32x4 x[XL ? 1 : U][MT][NX];
    };
    const char *xl = (const char *)lds + a.x_at;  // with XL: the lane's place in x
    {
        const int m = r < a.rows ? r : a.rows - 1;
        xl += m * a.x_row + g * XLANE * XS;
    }
    // Whole stages load without any condition: a branch would have the compiler
    // wait for the loads at its end. The last, part stage checks every piece.
    const int whole = a.k / (128 * U);
    auto load = [&](Stage &st, int c) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < U; ++u) st.w[u][t] = *(const u32x4 *)(wp[t] + (c * U + u) * 64);
        if constexpr (!XL)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < NX; ++j)
                        st.x[u][mt][j] = *(const u32x4 *)(xp[mt] + ((c * U + u) * 128 + j * XSTEP) * XS);
    };
    auto load_part = [&](Stage &st, int c) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k0 = (c * U + u) * 128;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                st.w[u][t] = u32x4{0, 0, 0, 0};
                if (k0 + g * 32 < a.k) st.w[u][t] = *(const u32x4 *)(wp[t] + k0 / 2);
            }
            if constexpr (!XL)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < NX; ++j) {
                        st.x[u][mt][j] = u32x4{0, 0, 0, 0};
                        if (k0 + (X8 ? g : j) * 32 < a.k)
                            st.x[u][mt][j] = *(const u32x4 *)(xp[mt] + (k0 + j * XSTEP) * XS);
                    }
        }
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[t][mt] = f32x4{0, 0, 0, 0};
    const uint32_t less2 = __is_same(E, __bf16) ? 0xc100c100u : 0xc800c800u;  // -8 of E, twice
    const E8 less = __builtin_bit_cast(E8, u32x4{less2, less2, less2, less2});

    const uint16_t *srow = (const uint16_t *)lds + (wn * NT * 16 + r) * a.scale_row;
    auto scale_of = [&](int t, int group) { return half_to_f32<E>(srow[t * 16 * a.scale_row + group]); };
    auto x_of = [&](const Stage &st, int c, int u, int mt, int j) {
        if constexpr (XL) return *(const u32x4 *)(xl + ((c * U + u) * 128 + j * XSTEP) * XS);
        else return st.x[u][mt][j];
    };
    auto chunk = [&](const Stage &st, int c, int u) {
        u32x4 w[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) w[t] = STAY ? st.w[u][t] : transpose_groups(st.w[u][t]);
        // e4m3 x: the words of the four products, low and high
        u32x4 xlo[MT], xhi[MT];
        if constexpr (X8) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const u32x4 p = x_of(st, c, u, mt, 0), q = x_of(st, c, u, mt, 1);
                xlo[mt] = u32x4{p[0], p[2], q[0], q[2]};
                xhi[mt] = u32x4{p[1], p[3], q[1], q[3]};
                if constexpr (!STAY) {
                    xlo[mt] = transpose_groups(xlo[mt]);
                    xhi[mt] = transpose_groups(xhi[mt]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            constexpr int J = GS / 32;  // products of a group
            E8 xf[MT][J];
            f32x4 sx[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                sx[mt] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if constexpr (X8) xf[mt][j] = order_x<E>(u32x2{xlo[mt][i * J + j], xhi[mt][i * J + j]});
                    else xf[mt][j] = order_x<E>(x_of(st, c, u, mt, i * J + j));
                    sx[mt] = mfma16(xf[mt][j], less, sx[mt]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float s = scale_of(t, c * GU + u * G + i);
                E8 wf[J];
#pragma unroll
                for (int j = 0; j < J; ++j) wf[j] = unpack<E>(w[t][i * J + j]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    f32x4 sum = sx[mt];
#pragma unroll
                    for (int j = 0; j < J; ++j) sum = mfma16(xf[mt][j], wf[j], sum);
                    acc[t][mt] += s * sum;
                }
            }
        }
    };

    auto compute = [&](const Stage &st, int c) {
#pragma unroll
        for (int u = 0; u < U; ++u) chunk(st, c, u);
    };

    Stage s0, s1;
    // this wave's stages follow each other
    const int first = wk * a.each;
    const int end = first + a.each < whole ? first + a.each : whole;
    const int n = end - first;
    auto at = [&](int i) { return first + i; };
    if (n > 0) load(s0, at(0));

    // Scales: a line of them serves many stages and would leave the first-level
    // cache in between, so they are brought to LDS once, 8 at a time.
    {
        const int pieces = (a.groups + 7) / 8;
        const int cols = a.wn * NT * 16, col0 = blockIdx.x * cols;
        for (int i = threadIdx.x; i < cols * pieces; i += blockDim.x) {
            const int col = i / pieces, g0 = (i - col * pieces) * 8;
            int64_t nn = col0 + col;
            nn = nn < a.n ? nn : a.n - 1;
            const Raw8<_Float16> v = load8<_Float16>((const _Float16 *)a.scales + nn * a.groups + g0, a.groups - g0);
            uint32_t *to = (uint32_t *)((uint16_t *)lds + col * a.scale_row + g0);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (g0 + 2 * q < a.scale_row) to[q] = v.w[q];
        }
        // groups that the last, part stage has beyond the row's
        const int stages = (a.k + 128 * U - 1) / (128 * U), stage_groups = stages * GU;
        for (int i = threadIdx.x; i < cols; i += blockDim.x)
            for (int q = a.groups; q < stage_groups; ++q) ((uint16_t *)lds)[i * a.scale_row + q] = 0;
        if constexpr (XL) {
            // x in pieces of 16 bytes, zeros past k
            const int row = stages * U * 128 * XS / 16;
            for (int i = threadIdx.x; i < a.rows * row; i += blockDim.x) {
                const int m = i / row, at = (i - m * row) * 16;
                u32x4 v = {0, 0, 0, 0};
                if (at < a.k * XS) v = *(const u32x4 *)((const char *)a.x + m * a.x_stride * XS + at);
                *(u32x4 *)((char *)lds + a.x_at + m * a.x_row + at) = v;
            }
        }
    }
    __syncthreads();

    // The next stage's loads are issued before this stage's products, and never
    // under a condition inside the loop (the compiler's waits count the
    // loads in flight on the path with the fewest).
    if (n > 0) {
        int i = 0;
        for (; i + 2 < n; i += 2) {
            load(s1, at(i + 1));
            compute(s0, at(i));
            load(s0, at(i + 2));
            compute(s1, at(i + 1));
        }
        if (i + 1 < n) {
            load(s1, at(i + 1));
            compute(s0, at(i));
            compute(s1, at(i + 1));
        } else {
            compute(s0, at(i));
        }
    }
    if (whole * U * 128 < a.k && whole / a.each == wk) {
        load_part(s0, whole);
        compute(s0, whole);
    }

    // Join the waves that share columns; lane: column r, rows 4g .. 4g + 3.
    __syncthreads();  // the scales have been read
    f32x4 *red = lds;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) red[(wave * NT * MT + t * MT + mt) * 64 + lane] = acc[t][mt];
    __syncthreads();
    for (int i = wk; i < NT * MT; i += a.wk) {
        f32x4 v = f32x4{0, 0, 0, 0};
        for (int q = 0; q < a.wk; ++q) v += red[((wn * a.wk + q) * NT * MT + i) * 64 + lane];
        const int64_t n = (int64_t)(tile0 + i / MT) * 16 + r;
        const int mb = m0 + (i % MT) * 16 + g * 4;
        if (n < a.n) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (mb + q < a.rows) {
                    const float f = X8 ? v[q] * a.x_scale[mb + q] : v[q];
                    ((uint16_t *)a.y)[(mb + q) * a.y_stride + n] = f32_to_half<E>(f);
                }
        }
    }
}

// Most LDS that x may take of a block (XL).
constexpr size_t kXLds = 40960;

template <typename E, bool X8, int GS, int NT, int MT> void go(Q4Args a, int wk, int wn, hipStream_t s) {
    // 128 bytes of each column a stage (a whole line) where the registers allow
    constexpr int U = NT * MT > 4 || (MT > 1 && NT > 1) ? 1 : 2;
    const int tiles = (a.n + 15) / 16;
    const int stages = (a.k + 128 * U - 1) / (128 * U);
    a.each = stages > wk ? (stages + wk - 1) / wk : 1;
    if (stages < wk * a.each) wk = stages > 0 ? (stages + a.each - 1) / a.each : 1;  // no wave without a stage
    a.wk = wk;
    a.wn = wn;
    // an odd number of words, so that the 16 columns of a tile read 16 banks
    a.scale_row = stages * U * 128 / GS;
    a.scale_row += a.scale_row % 2;
    if (a.scale_row / 2 % 2 == 0) a.scale_row += 2;
    const size_t scales = ((size_t)wn * NT * 16 * a.scale_row * 2 + 15) / 16 * 16;
    const size_t sums = (size_t)wk * wn * NT * MT * 1024;
    const dim3 grid((unsigned)((tiles + wn * NT - 1) / (wn * NT)), (unsigned)((a.rows + 16 * MT - 1) / (16 * MT)));
    if constexpr (MT == 1) {
        // rows 64 bytes apart in the banks: a tile's lanes read 64 bytes of each
        a.x_at = (int)scales;
        a.x_row = stages * U * 128 * (X8 ? 1 : 2) + 64;
        const size_t x = (size_t)a.rows * a.x_row;
        const size_t all = scales + x;
        if (x <= kXLds && all <= 65536) {
            q4_mfma<E, X8, GS, NT, MT, U, true><<<grid, 64 * wk * wn, all > sums ? all : sums, s>>>(a);
            return;
        }
    }
    q4_mfma<E, X8, GS, NT, MT, U, false><<<grid, 64 * wk * wn, scales > sums ? scales : sums, s>>>(a);
}

// Waves and tiles. A block reads all of its rows of x, which costs as much as the
// weights when x is 16 rows, and blocks beyond one a CU wait for a second turn. So
// a wave takes the fewest tiles of columns (1, 2 or 4) that leave at most 256
// blocks, and 4 where no number does; 8 waves share k, but 4 with 4 tiles of 32
// rows (their registers) or more than 256 blocks (two of them then run on a CU).
// Rows go in tiles of 16, or of 32 from 17 on; the weights are read again for every
// 32. Measured, us, on both sides (1, 2, 4 tiles a wave; bf16, k = 4096, groups of 128):
//   16 rows, 256 and 384 tiles of columns: 7.5, 8.3, 10.4 and 12.1, 8.5, 10.5;
//            512 and 768: 12.3, 8.7, 10.7 and 17.9, 14.2, 10.9;
//            4 tiles with 8 and 4 waves at 1024 and 2048: 11.3, 13.4 and 20.7, 19.6;
//   32 rows, 256 and 384: 11.1, 12.0, 15.4 and 20.0, 12.1, 15.3; 512 and 768: 20.2, 12.4, 15.6
//            and 28.9, 22.3, 16.0 (2 tiles with 4 waves at 256 and 512: 13.6, 14.4);
//   128 rows, 128 and 256: 20.0, 12.2, 15.5 and 36.6, 22.3, 15.8.
// (Tiles of 64 rows were slower at all sizes: 64 rows x 256, 896, 2048 tiles: 19, 39, 77 at
// their best against 12.6, 26, 50.) x that fits in LDS is cheap to share, and its blocks run
// several on a CU: one tile and 8 waves, from 1024 tiles on 2 x 4 waves of 2 tiles (1 row: 768
// tiles 9.3 and 9.6, 1024 11.4 and 10.4, 2048 19.5 and 15.2; 4 rows, 1024: 12.5 and 11.4).
// The scales of a block's columns fit in 64 KB of LDS: fewer tiles otherwise.
template <typename E, bool X8, int GS> void run(const Q4Args &a, hipStream_t s) {
    const int tiles = (a.n + 15) / 16;
    const int wide = (a.k / GS + 16) * 2 * 16;  // LDS bytes of a tile's scales
    if (a.rows <= 16 && (size_t)a.rows * ((a.k + 256) * (X8 ? 1 : 2) + 64) <= kXLds && wide * 4 <= 32768) {
        if (tiles >= 1024) go<E, X8, GS, 2, 1>(a, 4, 2, s);
        else go<E, X8, GS, 1, 1>(a, 8, 1, s);
        return;
    }
    const int64_t row_tiles = a.rows > 16 ? (a.rows + 31) / 32 : 1;
    auto one_turn = [&](int nt) { return (tiles + nt - 1) / nt * row_tiles <= 256; };
    int nt = one_turn(1) ? 1 : one_turn(2) ? 2 : 4;
    while (wide * nt > 65536) nt /= 2;
    if (a.rows > 16) {
        if (nt == 4) go<E, X8, GS, 4, 2>(a, 4, 1, s);
        else if (nt == 2) go<E, X8, GS, 2, 2>(a, 8, 1, s);
        else go<E, X8, GS, 1, 2>(a, 8, 1, s);
    } else {
        if (nt == 4) go<E, X8, GS, 4, 1>(a, one_turn(4) ? 8 : 4, 1, s);
        else if (nt == 2) go<E, X8, GS, 2, 1>(a, 8, 1, s);
        else go<E, X8, GS, 1, 1>(a, 8, 1, s);
    }
}

template <typename E> void run_type(const Q4Args &a, int x8, int64_t group, hipStream_t s) {
    if (x8) {
        if (group == 32) run<E, true, 32>(a, s);
        else if (group == 64) run<E, true, 64>(a, s);
        else run<E, true, 128>(a, s);
    } else {
        if (group == 32) run<E, false, 32>(a, s);
        else if (group == 64) run<E, false, 64>(a, s);
        else run<E, false, 128>(a, s);
    }
}

}  // namespace

hipError_t launch_q4_mfma(const convt_q4_problem &p, const void *x, const float *x_scale, const void *w,
                          const void *scales, void *y, hipStream_t stream) {
    const Q4Args a{x, w, scales, x_scale, y, p.x_stride, p.y_stride, (int32_t)p.rows, (int32_t)p.n, (int32_t)p.k,
                   (int32_t)(p.k / p.group), 0, 0, 0, 0, 0, 0};
    if (p.dtype == CONVT_DTYPE_BF16) run_type<__bf16>(a, p.x_quantised, p.group, stream);
    else run_type<_Float16>(a, p.x_quantised, p.group, stream);
    return hipGetLastError();
}

}  // namespace convt
