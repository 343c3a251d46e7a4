// Host checks that the C entry points over the cache share.
#pragma once

#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>

#include "decode.h"

namespace convt {

inline convt_status device_status(hipError_t e) { return e == hipSuccess ? CONVT_OK : CONVT_ERR_DEVICE; }

inline bool flag(int32_t v) { return v == 0 || v == 1; }

// CONVT_OK for an element type that the operators compute in.
inline convt_status check_dtype(int32_t dtype) {
    if (dtype == CONVT_DTYPE_F32 || dtype == CONVT_DTYPE_BF16 || dtype == CONVT_DTYPE_F16) return CONVT_OK;
    if (dtype == CONVT_DTYPE_I8 || dtype == CONVT_DTYPE_I32 || dtype == CONVT_DTYPE_I64) return CONVT_ERR_UNSUPPORTED;
    return CONVT_ERR_INVALID_ARGUMENT;
}

inline bool aligned(const void *p, uintptr_t n) { return (uintptr_t)p % n == 0; }

// Largest stride accepted: products with the indexes they go with stay far
// inside 63 bits.
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxIndex = ((int64_t)1 << 31) - 1;
// Most blocks of 256 threads along a grid's first axis (HIP counts an axis's
// threads in 32 bits).
constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;

// Strides of what is written are at least 1; what is only read may repeat (0).
inline bool strides_ok(const int64_t *s, int n, int64_t least = 1) {
    for (int i = 0; i < n; ++i)
        if (s[i] < least || s[i] > kMaxStride) return false;
    return true;
}

// Spacing of `width` elements' rows: at least the width, or, where they are
// only read, 0 (one row for all).
inline bool row_stride_ok(int64_t s, int64_t width, bool read) {
    return (s >= width && s <= kMaxStride) || (read && s == 0);
}

inline convt_status check_cache(const convt_cache_desc &c) {
    const convt_status st = check_dtype(c.dtype);
    if (st != CONVT_OK) return st;
    if (!flag(c.quantised) || c.reserved != 0) return CONVT_ERR_INVALID_ARGUMENT;
    if (c.n_pages < 0 || c.kv_heads < 1 || c.page_size < 1 || c.head_dim < 1) return CONVT_ERR_INVALID_ARGUMENT;
    if (c.n_pages > kMaxIndex || c.n_pages * (int64_t)c.page_size > kMaxIndex) return CONVT_ERR_INVALID_ARGUMENT;
    if (!strides_ok(c.k_stride, 3) || !strides_ok(c.v_stride, 3)) return CONVT_ERR_INVALID_ARGUMENT;
    if (c.head_dim > kMaxHeadDim) return CONVT_ERR_UNSUPPORTED;
    return CONVT_OK;
}

// The cache's own pointers: required unless it has no pages.
inline bool cache_pointers_ok(const convt_cache_desc &c, const void *k, const void *v, const void *ks, const void *vs) {
    if (c.quantised ? 0 : (ks || vs)) return false;
    if (c.n_pages == 0) return true;
    return k && v && (!c.quantised || (ks && vs));
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace convt
