// Products of a few rows with 4-bit weights and group scales on the matrix
// cores (two-byte element types, groups of 32, 64 or 128).
//
// Reading the weights bounds it (HBM), and next to that unpacking them: at 8
// TB/s a CU receives 26 weights a clock and has 64 vector lanes, so a weight
// may cost about two lane operations. The products run on unsigned values that
// cost less, with what they are too large by taken off as a multiple of sum x
// of the group; that is one more product, of x with a constant, whose result is
// where the group's sum starts. All products are exact in float32.
//   two-byte x: a weight w (0 .. 15) becomes the E value 16 + w by placing its
//     bits into the mantissa of 16.0, a shift and an and-or for two weights;
//     24 sum x is taken off. 16 + w keeps the sums within a factor of 6 of
//     those for w - 8: 2^-21 of the result against the 2^-8 or 2^-11 of its
//     rounding.
//   e4m3 x: the byte 0000wwww is the e4m3 value w * 2^-9, below and above the
//     normal range alike, so 8 weights take a shift and two ands, x stays in
//     8 bits, and 8 * 2^-9 sum x is taken off; the scale carries 2^9.
// One product serves up to 16 rows of x, and a group's scale multiplies its
// finished sum, once for 4 results.
//
// v_mfma_f32_16x16x32: A is 16 rows of x, B 16 columns (n) of W, a lane 8
// consecutive k of one. Loads of W are 16 bytes of one n a lane, 32 k, so that
// the four lanes of an n hold 128 k; each product wants its 32 k from four
// lanes, 8 each, so the words are transposed among the four lanes (4 lane
// swaps for 4 words) and every group of 32 k or more stays in one product.
// With e4m3 x and groups of 128 the product of 128 k takes the lanes' own 32 k.
// Unpacking leaves a word's weights in another order, to which x is brought by
// byte permutations; the sum does not mind.
//
// Waves of a block share columns with different k (WK of them, joined through
// LDS at the end) or take other columns (WN).
//
// Measured: 16 e4m3 rows x 8192 x 32768 (134 MB of weights): 33-36 us, 4 TB/s; its
// weights' loads alone 25, the products add 1, x (read by every block through
// the caches) the rest. One bf16 row: 32-34 us. One row x 4096 x 4096, 8.7 MB:
// 4.7 us, of which 2.5 are an empty launch and 2.5 a bare read of 8 MB.
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

constexpr int kMaxWaves = 8;

// 8 weights as 16 + w, in the order (0, 4), (1, 5), (2, 6), (3, 7).
template <typename E> __device__ __forceinline__ typename Vec8<E>::type unpack(uint32_t w) {
    u32x4 v;
    if constexpr (__is_same(E, __bf16)) {  // 7 mantissa bits: a weight at bits 3 .. 6
        v = u32x4{w << 3, w >> 1, w >> 5, w >> 9};
        for (int i = 0; i < 4; ++i) v[i] = (v[i] & 0x00780078u) | 0x41804180u;
    } else {  // 10 mantissa bits: bits 6 .. 9
        v = u32x4{w << 6, w << 2, w >> 2, w >> 6};
        for (int i = 0; i < 4; ++i) v[i] = (v[i] & 0x03c003c0u) | 0x4c004c00u;
    }
    return __builtin_bit_cast(typename Vec8<E>::type, v);
}

// 8 consecutive x in the same order.
template <typename E> __device__ __forceinline__ typename Vec8<E>::type order_x(u32x4 w) {
    return __builtin_bit_cast(typename Vec8<E>::type, u32x4{lo_pair(w[0], w[2]), hi_pair(w[0], w[2]),
                                                           lo_pair(w[1], w[3]), hi_pair(w[1], w[3])});
}

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma_e4m3(u32x2 a, u32x2 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0, 0, 0);
}
// both operands e4m3 (formats 0), unscaled
__device__ __forceinline__ f32x4 mfma_e4m3(i32x8 a, i32x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
// 8 weights as e4m3 w * 2^-9, in the order 0, 2, 4, 6, 1, 3, 5, 7; 8 consecutive
// codes of x in that order.
__device__ __forceinline__ u32x2 unpack_e4m3(uint32_t w) { return u32x2{w & 0x0f0f0f0fu, (w >> 4) & 0x0f0f0f0fu}; }
__device__ __forceinline__ u32x2 order_e4m3(uint32_t lo, uint32_t hi) {
    return u32x2{__builtin_amdgcn_perm(hi, lo, 0x06040200u), __builtin_amdgcn_perm(hi, lo, 0x07050301u)};
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
    constexpr bool WIDE = X8 && GS == 128;  // products of 128 k
    // x of a chunk: 4 pieces of 8 k for the products of 32 k, or 32 k in two
    typedef typename std::conditional<X8 && !WIDE, u32x2, u32x4>::type XW;
    constexpr int NX = WIDE ? 2 : 4;
    constexpr int XS = X8 ? 1 : 2;
    constexpr int XLANE = WIDE ? 32 : 8, XSTEP = WIDE ? 16 : 32;  // k between lane groups, between pieces
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
        XW x[XL ? 1 : U][MT][NX];
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
                        st.x[u][mt][j] = *(const XW *)(xp[mt] + ((c * U + u) * 128 + j * XSTEP) * XS);
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
                        st.x[u][mt][j] = XW{};
                        if (k0 + (WIDE ? 0 : j * 32) < a.k) st.x[u][mt][j] = *(const XW *)(xp[mt] + (k0 + j * XSTEP) * XS);
                    }
        }
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[t][mt] = f32x4{0, 0, 0, 0};
    // -24 of E, twice in a word; -8 * 2^-9 of e4m3, four times
    const uint32_t less = X8 ? 0x88888888u : __is_same(E, __bf16) ? 0xc1c0c1c0u : 0xce00ce00u;

    const uint16_t *srow = (const uint16_t *)lds + (wn * NT * 16 + r) * a.scale_row;
    auto scale_of = [&](int t, int group) { return half_to_f32<E>(srow[t * 16 * a.scale_row + group]); };
    auto x_of = [&](const Stage &st, int c, int u, int mt, int j) {
        if constexpr (XL) return *(const XW *)(xl + ((c * U + u) * 128 + j * XSTEP) * XS);
        else return st.x[u][mt][j];
    };
    auto chunk = [&](const Stage &st, int c, int u) {
        if constexpr (WIDE) {
            i32x8 xf[MT], off;
            f32x4 sx[MT];
#pragma unroll
            for (int i = 0; i < 8; ++i) off[i] = (int)less;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const XW x = x_of(st, c, u, mt, j);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const u32x2 v = order_e4m3(x[2 * i], x[2 * i + 1]);
                        xf[mt][4 * j + 2 * i] = (int)v[0];
                        xf[mt][4 * j + 2 * i + 1] = (int)v[1];
                    }
                }
                sx[mt] = mfma_e4m3(xf[mt], off, f32x4{0, 0, 0, 0});
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                i32x8 wf;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x2 v = unpack_e4m3(st.w[u][t][i]);
                    wf[2 * i] = (int)v[0];
                    wf[2 * i + 1] = (int)v[1];
                }
                const float s = scale_of(t, c * GU + u) * 512.0f;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) acc[t][mt] += s * mfma_e4m3(xf[mt], wf, sx[mt]);
            }
        } else {
            u32x4 w[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) w[t] = transpose_groups(st.w[u][t]);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                constexpr int J = GS / 32;  // products of a group
                typedef typename std::conditional<X8, u32x2, E8>::type F;
                F xf[MT][J];
                f32x4 sx[MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    sx[mt] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const XW x = x_of(st, c, u, mt, i * J + j);
                        if constexpr (X8) {
                            xf[mt][j] = order_e4m3(x[0], x[1]);
                            sx[mt] = mfma_e4m3(xf[mt][j], u32x2{less, less}, sx[mt]);
                        } else {
                            xf[mt][j] = order_x<E>(x);
                            sx[mt] = mfma16(xf[mt][j], __builtin_bit_cast(E8, u32x4{less, less, less, less}), sx[mt]);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float s = scale_of(t, c * GU + u * G + i) * (X8 ? 512.0f : 1.0f);
                    F wf[J];
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if constexpr (X8) wf[j] = unpack_e4m3(w[t][i * J + j]);
                        else wf[j] = unpack<E>(w[t][i * J + j]);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        f32x4 sum = sx[mt];
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            if constexpr (X8) sum = mfma_e4m3(xf[mt][j], wf[j], sum);
                            else sum = mfma16(xf[mt][j], wf[j], sum);
                        }
                        acc[t][mt] += s * sum;
                    }
                }
            }
        }
    };

    auto compute = [&](const Stage &st, int c) {
#pragma unroll
        for (int u = 0; u < U; ++u) chunk(st, c, u);
    };

    // The next stage's loads are issued before this stage's products, and never
    // under a condition inside the loop (the compiler's waits count the
    // loads in flight on the path with the fewest).
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
constexpr size_t kXLds = 32768;

template <typename E, bool X8, int GS, int NT, int MT> void go(Q4Args a, int wk, int wn, hipStream_t s) {
    // 128 bytes of each column a stage (a whole line) where the registers allow
    constexpr int U = NT * MT > 4 || MT == 4 || (MT > 1 && NT > 1) ? 1 : 2;
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

// Waves and tiles. Few columns: one tile a block and 8 waves over k, for as
// many blocks as there are CUs. Many columns: each block reads all of x, which
// costs as much as the weights when x is 16 rows (16 x 8192 e4m3 rows x
// 32768 columns: 33 us with 4 tiles a wave, 37 with 2, 42 with 1), so waves
// take more tiles. x that fits in LDS is cheap to share (1 x 8192 bf16 x
// 32768: 31 us from LDS with 2 tiles and 2 x 4 waves, 34 from the caches).
// The scales of a block's columns fit in 64 KB of LDS: fewer tiles otherwise.
template <typename E, bool X8, int GS> void run(const Q4Args &a, hipStream_t s) {
    const int tiles = (a.n + 15) / 16;
    const int wide = (a.k / GS + 16) * 2 * 16;  // LDS bytes of a tile's scales
    const bool four = wide * 4 <= 65536, two = wide * 2 <= 65536;
    if (a.rows > 32) {
        if (tiles >= 448 && two) go<E, X8, GS, 2, 4>(a, 4, 1, s);
        else go<E, X8, GS, 1, 4>(a, 8, 1, s);
    } else if (a.rows > 16) {
        if (tiles >= 1024 && four) go<E, X8, GS, 4, 2>(a, 4, 1, s);
        else if (tiles >= 448 && two) go<E, X8, GS, 2, 2>(a, 4, 1, s);
        else go<E, X8, GS, 1, 2>(a, 8, 1, s);
    } else if ((size_t)a.rows * a.k * (X8 ? 1 : 2) <= kXLds - 16 * 512 && wide * 4 <= 32768) {
        if (tiles >= 1024) go<E, X8, GS, 2, 1>(a, 4, 2, s);
        else go<E, X8, GS, 1, 1>(a, 8, 1, s);
    } else {
        if (tiles >= 1024 && four) go<E, X8, GS, 4, 1>(a, tiles >= 2048 ? 4 : 8, 1, s);
        else if (tiles >= 448 && two) go<E, X8, GS, 2, 1>(a, 8, 1, s);
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
