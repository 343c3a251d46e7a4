// Products of a few rows with 4-bit weights and group scales on the matrix
// cores (two-byte element types, groups of 32, 64 or 128).
//
// Reading the weights bounds it (HBM), and next to that unpacking them: at 8
// TB/s a CU receives 26 weights a clock and has 64 vector lanes, so a weight
// may cost about two lane operations. Hence:
//   - a weight w (0 .. 15) becomes the E value 16 + w by placing its bits into
//     the mantissa of 16.0: a shift and an and-or for two weights. The 24 that
//     are too much (16, and 8 for the sign) are taken off each group's sum as
//     24 sum x, and sum x is one more product, of x with ones, in the very
//     layout of the results. All products are exact in float32; 16 + w keeps
//     the sums within a factor of 6 of what they would be for w - 8, 2^-21 of
//     the result against the 2^-9 or 2^-12 of its rounding.
//   - one product serves up to 16 rows of x, and a group's scale multiplies its
//     finished sum, once for 4 results.
//
// v_mfma_f32_16x16x32: A is 16 rows of x, B 16 columns (n) of W, a lane 8
// consecutive k of one. Loads of W are 16 bytes of one n a lane, 32 k, so that
// the four lanes of an n hold 128 k; each product wants its 32 k from four
// lanes, 8 each, so the words are transposed among the four lanes (4 lane
// swaps for 4 words) and every group of 32 k or more stays in one product.
// The word's low and high halves hold k and k + 4 after unpacking, and x is
// brought to that order, which leaves the sum alone.
//
// Waves of a block share columns with different k (WK of them, joined through
// LDS at the end) or take other columns (WN).
#include "decode.h"
#include "kdecode.h"

namespace convt {

namespace {

struct Q4Args {
    const void *x, *w, *scales;
    const float *x_scale;
    void *y;
    int64_t x_stride, y_stride;
    int32_t rows, n, k, groups, chunks;  // chunks: 128 k each, the last may be part
    int32_t wk, wn;
};

constexpr int kMaxWaves = 8;

template <typename E> struct Vec8;
template <> struct Vec8<__bf16> { typedef bf16x8 type; };
template <> struct Vec8<_Float16> { typedef f16x8 type; };

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

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
template <typename E> __device__ __forceinline__ typename Vec8<E>::type order_x(u32x2 w) {
    // bytes (0, 4, 1, 5) and (2, 6, 3, 7), then two e4m3 codes at a time, exact
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
    if constexpr (__is_same(E, __bf16)) {
        typedef __bf16 e2 __attribute__((ext_vector_type(2)));
        const e2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true)};
        return bf16x8{v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]};
    } else {
        typedef _Float16 e2 __attribute__((ext_vector_type(2)));
        const e2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true),
                         __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true)};
        return f16x8{v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]};
    }
}

// Word j of lane group g <-> word g of lane group j (groups of 16 lanes).
__device__ __forceinline__ u32x4 transpose_groups(u32x4 w) {
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

template <typename E, bool X8, int GS, int NT, int MT>
__global__ __launch_bounds__(64 * kMaxWaves) void q4_mfma(Q4Args a) {
    typedef typename Vec8<E>::type E8;
    typedef typename std::conditional<X8, u32x2, u32x4>::type XW;
    constexpr int XS = X8 ? 1 : 2;
    constexpr int G = 128 / GS;  // groups of a chunk
    __shared__ f32x4 red[kMaxWaves][NT * MT][64];
    const int lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wk = wave % a.wk, wn = wave / a.wk;
    const int m0 = blockIdx.y * 16 * MT;
    const int tile0 = (blockIdx.x * a.wn + wn) * NT;  // first tile of 16 columns

    const char *wp[NT];
    const uint16_t *sp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        // columns past the last read the last one and are not stored
        int64_t n = (int64_t)(tile0 + t) * 16 + r;
        n = n < a.n ? n : a.n - 1;
        wp[t] = (const char *)a.w + n * (a.k / 2) + g * 16;
        sp[t] = (const uint16_t *)a.scales + n * a.groups;
    }
    const char *xp[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) xp[mt] = (const char *)a.x + ((m0 + mt * 16 + r) * a.x_stride + g * 8) * XS;

    struct Stage {
        u32x4 w[NT];
        XW x[MT][4];
        uint16_t s[NT][G];
    };
    auto load = [&](Stage &st, int c) {
        const int k0 = c * 128;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            st.w[t] = u32x4{0, 0, 0, 0};
            if (k0 + g * 32 < a.k) st.w[t] = *(const u32x4 *)(wp[t] + k0 / 2);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                st.x[mt][j] = XW{};
                if (m0 + mt * 16 + r < a.rows && k0 + j * 32 < a.k) st.x[mt][j] = *(const XW *)(xp[mt] + (k0 + j * 32) * XS);
            }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int at = c * G + i;
                st.s[t][i] = sp[t][at < a.groups ? at : a.groups - 1];
            }
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[t][mt] = f32x4{0, 0, 0, 0};
    const uint32_t one2 = __is_same(E, __bf16) ? 0x3f803f80u : 0x3c003c00u;
    const E8 ones = __builtin_bit_cast(E8, u32x4{one2, one2, one2, one2});

    auto compute = [&](const Stage &st) {
        u32x4 w[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) w[t] = transpose_groups(st.w[t]);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            f32x4 sum[NT][MT], sx[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                sx[mt] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < NT; ++t) sum[t][mt] = f32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int jj = 0; jj < GS / 32; ++jj) {
                const int j = i * (GS / 32) + jj;
                E8 xf[MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    xf[mt] = order_x<E>(st.x[mt][j]);
                    sx[mt] = mfma16(xf[mt], ones, sx[mt]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const E8 wf = unpack<E>(w[t][j]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) sum[t][mt] = mfma16(xf[mt], wf, sum[t][mt]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float s = half_to_f32<E>(st.s[t][i]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[t][mt][q] += s * (sum[t][mt][q] - 24.0f * sx[mt][q]);
            }
        }
    };

    Stage s0, s1;
    int c = wk;
    if (c < a.chunks) load(s0, c);
    while (c < a.chunks) {
        if (c + a.wk < a.chunks) load(s1, c + a.wk);
        compute(s0);
        c += a.wk;
        if (c >= a.chunks) break;
        if (c + a.wk < a.chunks) load(s0, c + a.wk);
        compute(s1);
        c += a.wk;
    }

    // Join the waves that share columns; lane: column r, rows 4g .. 4g + 3.
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) red[wave][t * MT + mt][lane] = acc[t][mt];
    __syncthreads();
    for (int i = wk; i < NT * MT; i += a.wk) {
        f32x4 v = f32x4{0, 0, 0, 0};
        for (int q = 0; q < a.wk; ++q) v += red[wn * a.wk + q][i][lane];
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

template <typename E, bool X8, int GS, int NT, int MT> void go(Q4Args &a, hipStream_t s) {
    const int tiles = (a.n + 15) / 16;
    const dim3 grid((unsigned)((tiles + a.wn * NT - 1) / (a.wn * NT)), (unsigned)((a.rows + 16 * MT - 1) / (16 * MT)));
    q4_mfma<E, X8, GS, NT, MT><<<grid, 64 * a.wk * a.wn, 0, s>>>(a);
}

template <typename E, bool X8, int GS> void run(Q4Args &a, hipStream_t s) {
    const int tiles = (a.n + 15) / 16;
    a.wk = 8;
    a.wn = 1;
    if (a.rows > 32) go<E, X8, GS, 1, 4>(a, s);
    else if (a.rows > 16) go<E, X8, GS, 1, 2>(a, s);
    else if (tiles >= 1024) go<E, X8, GS, 2, 1>(a, s);
    else go<E, X8, GS, 1, 1>(a, s);
}

template <typename E> void run_type(Q4Args &a, int x8, int64_t group, hipStream_t s) {
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
    Q4Args a{x, w, scales, x_scale, y, p.x_stride, p.y_stride, (int32_t)p.rows, (int32_t)p.n, (int32_t)p.k,
             (int32_t)(p.k / p.group), (int32_t)((p.k + 127) / 128), 0, 0};
    if (p.dtype == CONVT_DTYPE_BF16) run_type<__bf16>(a, p.x_quantised, p.group, stream);
    else run_type<_Float16>(a, p.x_quantised, p.group, stream);
    return hipGetLastError();
}

}  // namespace convt
