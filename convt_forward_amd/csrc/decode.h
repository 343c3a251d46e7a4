// Parameters and launchers of the decoding-step kernels (host side: checked
// in decode_api.cpp before any launch). Plain data and launch statuses only.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "convt_decode.h"
#include "convt_internal.h"

namespace convt {

// The multiplier of fast_div for a divisor d >= 1 (see FastDiv).
inline FastDiv divisor_of(uint32_t d) {
    uint32_t s = 0;
    while (((uint64_t)1 << s) < d) ++s;
    const uint64_t m = (((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1;
    return FastDiv{(uint32_t)m, s};
}

// Most head dimensions a cache row may have: 64 lanes of 8 elements.
constexpr int kMaxHeadDim = 512;

hipError_t launch_rms_norm(const convt_rms_norm_problem &p, const void *x, const void *weight,
                           const void *residual, void *y, float *scale, void *residual_out,
                           hipStream_t stream);

struct CacheArgs {
    const void *k, *v;            // rows in the element type (written by a read)
    void *k_cache, *v_cache;
    float *k_scale, *v_scale;
    const int64_t *slots;
    int64_t row_stride[2][2];     // [k, v][token, head]
    int64_t cache_stride[2][3];   // [k, v][page, head, token]
    int64_t n_slots;              // n_pages * page_size
    int64_t tokens;
    uint32_t items;               // blocks of tokens * kv_heads (k_cache.hip)
    int32_t kv_heads, page_size, head_dim;
    FastDiv div_heads, div_page;
};
// write = 0 reads the cache into k and v
hipError_t launch_cache(const CacheArgs &a, int dtype, int quantised, int write, hipStream_t stream);

struct AttendArgs {
    const void *q, *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *page_table, *lengths;
    void *out;
    float *lse;
    float *part_o, *part_ml;      // workspace: [batch * heads][chunks][head_dim], [..][chunks][2]
    int64_t q_stride[2], out_stride[2];
    int64_t k_stride[3], v_stride[3];
    int64_t table_stride, n_pages;
    int32_t batch, heads, kv_heads, share;  // share = heads / kv_heads
    int32_t head_dim, page_size, max_length;
    int32_t chunks, chunk_tokens;
    float scale_log2e;            // scale * log2(e): the softmax runs on powers of two
    FastDiv div_page, div_heads;
};
hipError_t launch_attend_direct(const AttendArgs &a, int dtype, int quantised, hipStream_t stream);
hipError_t launch_attend_mfma(const AttendArgs &a, int dtype, int quantised, hipStream_t stream);
hipError_t launch_attend_join(const AttendArgs &a, int dtype, hipStream_t stream);

hipError_t launch_q4_direct(const convt_q4_problem &p, const void *x, const float *x_scale, const void *w,
                            const void *scales, void *y, hipStream_t stream);
hipError_t launch_q4_mfma(const convt_q4_problem &p, const void *x, const float *x_scale, const void *w,
                          const void *scales, void *y, hipStream_t stream);

}  // namespace convt
