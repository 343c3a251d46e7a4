// Writing tokens' keys and values into the paged cache, and reading them back.
//
// One (token, head) row is handled by a power of two of lanes, 8 elements
// each, so that a wave moves several whole rows with wide accesses and the
// row's largest magnitude is a reduction over neighbouring lanes. Memory
// traffic bounds both: each element is read once and written once.
#include "decode.h"
#include "kdecode.h"

namespace convt {

namespace {

// (page, head, token) place of row `item` of the tokens x heads rows, or
// false if its slot lies outside the cache.
struct Place {
    uint32_t token, head, page, off;
};
__device__ __forceinline__ bool place_of(const CacheArgs &a, uint32_t item, Place &p) {
    p.token = fast_div(item, a.div_heads);
    p.head = item - p.token * (uint32_t)a.kv_heads;
    const int64_t slot = a.slots[p.token];
    if (slot < 0 || slot >= a.n_slots) return false;
    p.page = fast_div((uint32_t)slot, a.div_page);
    p.off = (uint32_t)slot - p.page * (uint32_t)a.page_size;
    return true;
}
__device__ __forceinline__ int64_t cache_offset(const int64_t *stride, const Place &p) {
    return p.page * stride[0] + p.head * stride[1] + p.off * stride[2];
}
__device__ __forceinline__ int64_t scale_offset(const CacheArgs &a, const Place &p) {
    return ((int64_t)p.page * a.kv_heads + p.head) * a.page_size + p.off;
}

// blockIdx.y: 0 keys, 1 values. lanes = 1 << lanes_log2 lanes per row.
template <typename T, bool Q>
__global__ __launch_bounds__(256) void write_kernel(CacheArgs a, int lanes_log2) {
    const int kv = blockIdx.y;
    const int piece = (threadIdx.x & ((1 << lanes_log2) - 1)) * 8;
    const int rows = 256 >> lanes_log2;
    const T *src = (const T *)(kv ? a.v : a.k);
    // every lane of a row takes the same way, and so do all lanes of the
    // block up to the last rows: `item` is clamped there, not left out
    for (uint64_t base = (uint64_t)blockIdx.x * rows; base < a.items; base += (uint64_t)gridDim.x * rows) {
        const uint64_t item = base + (threadIdx.x >> lanes_log2);
        Place p;
        const bool in = item < a.items && place_of(a, (uint32_t)item, p);
        const int n = in ? a.head_dim - piece : 0;
        float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        Raw8<T> raw = zero8<T>();
        if (n > 0) raw = load8<T>(src + p.token * a.row_stride[kv][0] + p.head * a.row_stride[kv][1] + piece, n);
        raw_to_f32<T>(raw, f);
        if constexpr (Q) {
            uint32_t amax = 0;
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = abs_bits(f[j]);
                amax = b > amax ? b : amax;
            }
            for (int m = 1; m < (1 << lanes_log2); m <<= 1) {
                const uint32_t o = (uint32_t)__shfl_xor((int)amax, m);
                amax = o > amax ? o : amax;
            }
            float inv;
            const float s = row_scale(amax, inv);
            for (int j = 0; j < 8; ++j) f[j] *= inv;
            if (n > 0) {
                store8_e4m3((uint8_t *)(kv ? a.v_cache : a.k_cache) + cache_offset(a.cache_stride[kv], p) + piece, f, n);
                if (piece == 0) (kv ? a.v_scale : a.k_scale)[scale_offset(a, p)] = s;
            }
        } else if (n > 0) {
            store8<T>((T *)(kv ? a.v_cache : a.k_cache) + cache_offset(a.cache_stride[kv], p) + piece, f, n);
        }
    }
}

template <typename T, bool Q>
__global__ __launch_bounds__(256) void read_kernel(CacheArgs a, int lanes_log2) {
    const int kv = blockIdx.y;
    const int piece = (threadIdx.x & ((1 << lanes_log2) - 1)) * 8;
    const int rows = 256 >> lanes_log2;
    T *dst = (T *)(kv ? a.v : a.k);
    const int n = a.head_dim - piece;
    if (n <= 0) return;
    for (uint64_t item = (uint64_t)blockIdx.x * rows + (threadIdx.x >> lanes_log2); item < a.items;
         item += (uint64_t)gridDim.x * rows) {
        Place p;
        float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (place_of(a, (uint32_t)item, p)) {
            const int64_t at = cache_offset(a.cache_stride[kv], p) + piece;
            if constexpr (Q) {
                const float s = (kv ? a.v_scale : a.k_scale)[scale_offset(a, p)];
                e4m3_to_f32(load8_e4m3((const uint8_t *)(kv ? a.v_cache : a.k_cache) + at, n), f);
                for (int j = 0; j < 8; ++j) f[j] *= s;
            } else {
                raw_to_f32<T>(load8<T>((const T *)(kv ? a.v_cache : a.k_cache) + at, n), f);
            }
        }
        store8<T>(dst + p.token * a.row_stride[kv][0] + p.head * a.row_stride[kv][1] + piece, f, n);
    }
}

template <typename T, bool Q> void run(const CacheArgs &a, int write, hipStream_t s) {
    int lanes_log2 = 0;
    while ((8 << lanes_log2) < a.head_dim) ++lanes_log2;
    const uint64_t rows = 256 >> lanes_log2;
    const uint64_t blocks = (a.items + rows - 1) / rows;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)), 2);
    if (write) write_kernel<T, Q><<<grid, 256, 0, s>>>(a, lanes_log2);
    else read_kernel<T, Q><<<grid, 256, 0, s>>>(a, lanes_log2);
}

template <typename T> void run_type(const CacheArgs &a, int quantised, int write, hipStream_t s) {
    if (quantised) run<T, true>(a, write, s);
    else run<T, false>(a, write, s);
}

}  // namespace

hipError_t launch_cache(const CacheArgs &a, int dtype, int quantised, int write, hipStream_t stream) {
    if (dtype == CONVT_DTYPE_F32) run_type<float>(a, quantised, write, stream);
    else if (dtype == CONVT_DTYPE_BF16) run_type<uint16_t>(a, quantised, write, stream);
    else run_type<_Float16>(a, quantised, write, stream);
    return hipGetLastError();
}

}  // namespace convt
