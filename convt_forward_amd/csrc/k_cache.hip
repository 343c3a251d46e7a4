// Writing tokens' keys and values into the paged cache, and reading them back.
//
// One (token, head) row is handled by a power of two of lanes, 8 elements
// each, so that a wave moves several whole rows with wide accesses and the
// row's largest magnitude is a reduction over neighbouring lanes. A lane takes
// the rows of kTokens neighbouring tokens of one head: their slots, then
// their elements are requested together, where one row after the other would
// wait twice for memory each; neighbouring tokens lie next to each other in
// the cache, the heads of a token in the rows outside it, so both sides come
// in pieces of several rows.
// Memory traffic bounds both directions: each element is read once and
// written once. Measured: 32767 tokens x 8 heads x 128 written, f16 to e4m3, 204 MB:
// 41 us, 4.9 TB/s, the rate of a large copy; 65536 tokens read from e4m3 to bf16, 407
// MB: 77 us, 5.3 TB/s; 64 tokens written: 3.2 us a call of a graph, 4.1 in a
// kernel trace (one row a lane, its load and store alone: 51 and 97 us for the
// large ones, 2.7 for the small).
#include "decode.h"
#include "kdecode.h"

namespace convt {

namespace {

constexpr int kTokens = 4;

// The lane's piece of a row. FULL: lanes past the row read its first piece.
template <typename T, bool FULL> __device__ __forceinline__ Raw8<T> load_piece(const T *row, int piece, int n) {
    if constexpr (FULL) {
        Raw8<T> r = load8<T>(row + (n > 0 ? piece : 0), 8);
        if (n <= 0) r = zero8<T>();
        return r;
    } else {
        return n > 0 ? load8<T>(row + piece, n) : zero8<T>();
    }
}
template <bool FULL> __device__ __forceinline__ u32x2 load_codes(const uint8_t *row, int piece, int n) {
    return load8_e4m3(row + piece, FULL ? 8 : n);
}

// blockIdx.y: 0 keys, 1 values. 1 << lanes_log2 lanes a row. FULL: head_dim is
// a multiple of 8, so that no lane has part of a piece.
template <typename T, bool Q, bool FULL>
__global__ __launch_bounds__(256) void write_kernel(CacheArgs a, int lanes_log2) {
    const int kv = blockIdx.y;
    const int piece = (threadIdx.x & ((1 << lanes_log2) - 1)) * 8;
    const int rows = 256 >> lanes_log2;
    const int n = FULL ? (piece < a.head_dim ? 8 : 0) : a.head_dim - piece;
    const T *src = (const T *)(kv ? a.v : a.k);
    // all lanes of a wave stay in the loop together, for the reduction
    for (uint64_t base = (uint64_t)blockIdx.x * rows; base < a.items; base += (uint64_t)gridDim.x * rows) {
        // Rows past the last read the last one and are not stored: loads
        // under a condition would each be waited for at its end.
        const uint64_t at = base + (threadIdx.x >> lanes_log2);
        const uint32_t item = at < a.items ? (uint32_t)at : a.items - 1;
        const uint32_t block = fast_div(item, a.div_heads);
        const uint32_t head = item - block * (uint32_t)a.kv_heads;
        int64_t slot[kTokens];
        Raw8<T> raw[kTokens];
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            const int64_t t = (int64_t)block * kTokens + i;
            const int64_t tc = t < a.tokens ? t : a.tokens - 1;
            slot[i] = a.slots[tc];
            raw[i] = load_piece<T, FULL>(src + tc * a.row_stride[kv][0] + head * a.row_stride[kv][1], piece, n);
        }
        Place p[kTokens];
#pragma unroll
        for (int i = 0; i < kTokens; ++i)
            p[i] = place_of(a, at < a.items && (int64_t)block * kTokens + i < a.tokens ? slot[i] : -1);
        float f[kTokens][8];
        uint32_t amax[kTokens];
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            raw_to_f32<T>(raw[i], f[i]);
            amax[i] = 0;
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = abs_bits(f[i][j]);
                amax[i] = b > amax[i] ? b : amax[i];
            }
        }
        if constexpr (Q) group_max_u32(amax, lanes_log2);
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            if constexpr (Q) {
                float inv;
                const float s = row_scale(amax[i], inv);
                for (int j = 0; j < 8; ++j) f[i][j] *= inv;
                if (p[i].page >= 0 && n > 0) {
                    store8_e4m3((uint8_t *)(kv ? a.v_cache : a.k_cache) + cache_offset(a.cache_stride[kv], head, p[i]) + piece, f[i], n);
                    if (piece == 0) (kv ? a.v_scale : a.k_scale)[scale_offset(a, head, p[i])] = s;
                }
            } else if (p[i].page >= 0 && n > 0) {
                store8<T>((T *)(kv ? a.v_cache : a.k_cache) + cache_offset(a.cache_stride[kv], head, p[i]) + piece, f[i], n);
            }
        }
    }
}

template <typename T, bool Q, bool FULL>
__global__ __launch_bounds__(256) void read_kernel(CacheArgs a, int lanes_log2) {
    const int kv = blockIdx.y;
    const int piece = (threadIdx.x & ((1 << lanes_log2) - 1)) * 8;
    const int rows = 256 >> lanes_log2;
    T *dst = (T *)(kv ? a.v : a.k);
    const int n = FULL ? (piece < a.head_dim ? 8 : 0) : a.head_dim - piece;
    if (n <= 0) return;
    for (uint64_t item = (uint64_t)blockIdx.x * rows + (threadIdx.x >> lanes_log2); item < a.items;
         item += (uint64_t)gridDim.x * rows) {
        const uint32_t block = fast_div((uint32_t)item, a.div_heads);
        const uint32_t head = (uint32_t)item - block * (uint32_t)a.kv_heads;
        Place p[kTokens];
        int64_t slot[kTokens];
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            const int64_t t = (int64_t)block * kTokens + i;
            slot[i] = a.slots[t < a.tokens ? t : a.tokens - 1];
        }
        typedef typename std::conditional<Q, u32x2, Raw8<T>>::type Cell;
        Cell raw[kTokens];
        float s[kTokens];
#pragma unroll
        for (int i = 0; i < kTokens; ++i) p[i] = place_of(a, slot[i]);
        if (a.n_slots > 0) {
#pragma unroll
            for (int i = 0; i < kTokens; ++i) {
                // a slot outside reads the first place, to be dropped
                const Place q = p[i].page < 0 ? Place{0, 0} : p[i];
                const int64_t at = cache_offset(a.cache_stride[kv], head, q);
                if constexpr (Q) {
                    s[i] = (kv ? a.v_scale : a.k_scale)[scale_offset(a, head, q)];
                    raw[i] = load_codes<FULL>((const uint8_t *)(kv ? a.v_cache : a.k_cache) + at, piece, n);
                } else {
                    raw[i] = load_piece<T, FULL>((const T *)(kv ? a.v_cache : a.k_cache) + at, piece, n);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            const int64_t t = (int64_t)block * kTokens + i;
            if (t >= a.tokens) continue;
            float f[8];
            if constexpr (Q) {
                e4m3_to_f32(raw[i], f);
                for (int j = 0; j < 8; ++j) f[j] *= s[i];
            } else {
                raw_to_f32<T>(raw[i], f);
            }
            for (int j = 0; j < 8; ++j) f[j] = p[i].page < 0 ? 0.0f : f[j];
            store8<T>(dst + t * a.row_stride[kv][0] + head * a.row_stride[kv][1] + piece, f, n);
        }
    }
}

template <typename T, bool Q, bool FULL> void go(const CacheArgs &a, int write, int lanes_log2, hipStream_t s) {
    const uint64_t rows = 256 >> lanes_log2;
    const uint64_t blocks = (a.items + rows - 1) / rows;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)), 2);
    if (write) write_kernel<T, Q, FULL><<<grid, 256, 0, s>>>(a, lanes_log2);
    else read_kernel<T, Q, FULL><<<grid, 256, 0, s>>>(a, lanes_log2);
}

template <typename T, bool Q> void run(CacheArgs a, int write, hipStream_t s) {
    int lanes_log2 = 0;
    while ((8 << lanes_log2) < a.head_dim) ++lanes_log2;
    a.items = (uint32_t)((a.tokens + kTokens - 1) / kTokens * a.kv_heads);
    if (a.head_dim % 8 == 0) go<T, Q, true>(a, write, lanes_log2, s);
    else go<T, Q, false>(a, write, lanes_log2, s);
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
