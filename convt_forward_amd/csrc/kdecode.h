// Device helpers of the decoding-step kernels: loads and stores of 8 elements
// at any alignment, e4m3 conversion, and wave reductions.
#pragma once

#include <type_traits>

#include "decode.h"
#include "kcommon.h"

namespace convt {

// Vector words at the alignment of one element: gfx950 takes global accesses
// at any byte address, so odd row strides and odd widths keep wide loads.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// One word of two two-byte elements as float32.
template <typename T> __device__ __forceinline__ void word_to_f32(uint32_t w, float &a, float &b);
template <> __device__ __forceinline__ void word_to_f32<uint16_t>(uint32_t w, float &a, float &b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
}
template <> __device__ __forceinline__ void word_to_f32<_Float16>(uint32_t w, float &a, float &b) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    const h2 h = __builtin_bit_cast(h2, w);
    a = (float)h[0];
    b = (float)h[1];
}

// The arithmetic type of a two-byte element type's bit pattern.
template <typename T> struct Arith { typedef T type; };
template <> struct Arith<uint16_t> { typedef __bf16 type; };

// 8 elements of an arithmetic type, an operand of the 16 x 16 x 32 products.
template <typename E> struct Vec8;
template <> struct Vec8<__bf16> { typedef bf16x8 type; };
template <> struct Vec8<_Float16> { typedef f16x8 type; };

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Two e4m3 codes (the low or high half of a word) as two E in a word, times a
// power of two, exact.
template <typename E, bool HI> __device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, float scale = 1.0f) {
    if constexpr (__is_same(E, __bf16))
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HI));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, HI));
}

// Two bfloat16 values with infinities (and NaN) replaced by the largest finite
// value of their sign, as integers: unsigned, that bounds the negative ones;
// signed, the positive ones.
__device__ __forceinline__ uint32_t finite_bf16(uint32_t w) {
    typedef uint16_t u2 __attribute__((ext_vector_type(2)));
    typedef int16_t i2 __attribute__((ext_vector_type(2)));
    const u2 n = __builtin_elementwise_min(__builtin_bit_cast(u2, w), u2{0xff7f, 0xff7f});
    const i2 v = __builtin_elementwise_min(__builtin_bit_cast(i2, n), i2{0x7f7f, 0x7f7f});
    return __builtin_bit_cast(uint32_t, v);
}

// 8 elements in the registers they are loaded into.
template <typename T> struct Raw8 { u32x4 w; };
template <> struct Raw8<float> { f32x4 lo, hi; };

// n (1 .. 8) elements at p; the rest are zero.
template <typename T> __device__ __forceinline__ Raw8<T> load8(const T *p, int n) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
        if (n >= 8) {
            r.lo = *(const f32x4_a4 *)p;
            r.hi = *(const f32x4_a4 *)(p + 4);
        } else {
            r.lo = r.hi = f32x4{0, 0, 0, 0};
            for (int i = 0; i < 4; ++i) {
                if (i < n) r.lo[i] = p[i];
                if (i + 4 < n) r.hi[i] = p[i + 4];
            }
        }
    } else {
        if (n >= 8) {
            r.w = *(const u32x4_a2 *)p;
        } else {
            const uint16_t *u = (const uint16_t *)p;
            for (int i = 0; i < 4; ++i) {
                uint32_t w = 0;
                if (2 * i < n) w = u[2 * i];
                if (2 * i + 1 < n) w |= (uint32_t)u[2 * i + 1] << 16;
                r.w[i] = w;
            }
        }
    }
    return r;
}

template <typename T> __device__ __forceinline__ Raw8<T> zero8() {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4)
        r.lo = r.hi = f32x4{0, 0, 0, 0};
    else
        r.w = u32x4{0, 0, 0, 0};
    return r;
}

template <typename T> __device__ __forceinline__ void raw_to_f32(const Raw8<T> &r, float *f) {
    if constexpr (sizeof(T) == 4) {
        for (int i = 0; i < 4; ++i) {
            f[i] = r.lo[i];
            f[i + 4] = r.hi[i];
        }
    } else {
        for (int i = 0; i < 4; ++i) word_to_f32<T>(r.w[i], f[2 * i], f[2 * i + 1]);
    }
}

// The first n (1 .. 8) of f, rounded to T (nearest even), at p.
template <typename T> __device__ __forceinline__ void store8(T *p, const float *f, int n) {
    if constexpr (sizeof(T) == 4) {
        if (n >= 8) {
            *(f32x4_a4 *)p = f32x4{f[0], f[1], f[2], f[3]};
            *(f32x4_a4 *)(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
        } else {
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = f[i];
        }
    } else {
        typedef typename Arith<T>::type E;
        u32x4 w;
        for (int i = 0; i < 4; ++i) w[i] = pack_half2<E>(f[2 * i], f[2 * i + 1]);
        if (n >= 8) {
            *(u32x4_a2 *)p = w;
        } else {
            uint16_t *u = (uint16_t *)p;
            for (int i = 0; i < 8; ++i)
                if (i < n) u[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        }
    }
}

// e4m3 codes of 8 values (nearest even; the values are at most 448 by the
// choice of the scale, NaN stays NaN), the first n of them stored at p.
__device__ __forceinline__ void store8_e4m3(uint8_t *p, const float *f, int n) {
    u32x2 w;
    for (int i = 0; i < 2; ++i) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
        w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], v, true);
    }
    if (n >= 8) {
        *(u32x2_a1 *)p = w;
    } else {
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
    }
}

// n (1 .. 8) e4m3 codes at p in two words; the rest are code 0 (zero).
__device__ __forceinline__ u32x2 load8_e4m3(const uint8_t *p, int n) {
    if (n >= 8) return *(const u32x2_a1 *)p;
    u32x2 w = {0, 0};
    for (int i = 0; i < 8; ++i)
        if (i < n) w[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
    return w;
}
__device__ __forceinline__ void e4m3_to_f32(u32x2 w, float *f) {
    for (int i = 0; i < 2; ++i) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        f[4 * i] = a[0];
        f[4 * i + 1] = a[1];
        f[4 * i + 2] = b[0];
        f[4 * i + 3] = b[1];
    }
}

// |v| as an integer that orders like it, with NaN above infinity: the
// maximum of these carries a NaN that a floating maximum would drop.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale of a row from the bits of its largest magnitude, and 1 / scale.
// The lower limit 2^-126 keeps the reciprocal finite and a row of zeros zero;
// a NaN passes it.
__device__ __forceinline__ float row_scale(uint32_t amax_bits, float &inv) {
    float s = __uint_as_float(amax_bits) / 448.0f;
    if (s < 0x1p-126f) s = 0x1p-126f;
    inv = 1.0f / s;
    return s;
}

// Place of a slot in the cache; page < 0 if it lies outside.
struct Place {
    int32_t page, off;
};
__device__ __forceinline__ Place place_of(const CacheArgs &a, int64_t slot) {
    if (slot < 0 || slot >= a.n_slots) return Place{-1, 0};
    const uint32_t page = fast_div((uint32_t)slot, a.div_page);
    return Place{(int32_t)page, (int32_t)((uint32_t)slot - page * (uint32_t)a.page_size)};
}
__device__ __forceinline__ int64_t cache_offset(const int64_t *stride, uint32_t head, const Place &p) {
    return p.page * stride[0] + head * stride[1] + p.off * stride[2];
}
__device__ __forceinline__ int64_t scale_offset(const CacheArgs &a, uint32_t head, const Place &p) {
    return ((int64_t)p.page * a.kv_heads + head) * a.page_size + p.off;
}

// The largest over the 1 << log2 neighbouring lanes of each of N values,
// given to all of them: lane exchanges inside rows of 16 lanes by DPP, between
// rows by the row swaps.
template <int CTRL> __device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
    return o > v ? o : v;
}
template <int N> __device__ __forceinline__ void group_max_u32(uint32_t (&v)[N], int log2) {
    if (log2 > 0)
        for (int i = 0; i < N; ++i) v[i] = max_dpp<0xb1>(v[i]);  // quad_perm 1, 0, 3, 2
    if (log2 > 1)
        for (int i = 0; i < N; ++i) v[i] = max_dpp<0x4e>(v[i]);  // quad_perm 2, 3, 0, 1
    if (log2 > 2)
        for (int i = 0; i < N; ++i) v[i] = max_dpp<0x141>(v[i]);  // row_half_mirror
    if (log2 > 3)
        for (int i = 0; i < N; ++i) v[i] = max_dpp<0x140>(v[i]);  // row_mirror
    if (log2 > 4)
        for (int i = 0; i < N; ++i) {
            auto a = __builtin_amdgcn_permlane16_swap(v[i], v[i], false, false);
            v[i] = a[0] > a[1] ? a[0] : a[1];
        }
    if (log2 > 5)
        for (int i = 0; i < N; ++i) {
            auto a = __builtin_amdgcn_permlane32_swap(v[i], v[i], false, false);
            v[i] = a[0] > a[1] ? a[0] : a[1];
        }
}

// The same exchanges for a float's sum or largest over the wave.
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0xb1>(v);
    v += dpp<0x4e>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp<0xb1>(v));
    v = fmaxf(v, dpp<0x4e>(v));
    v = fmaxf(v, dpp<0x141>(v));
    v = fmaxf(v, dpp<0x140>(v));
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    uint32_t a[1] = {v};
    group_max_u32(a, 6);
    return a[0];
}

}  // namespace convt
