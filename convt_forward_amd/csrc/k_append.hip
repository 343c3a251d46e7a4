// Rotary positions and the cache write of new tokens in one pass: q rotated
// into q_out, k rotated and v as it is into the paged cache.
//
// A block takes a few tokens: it first forms sine and cosine of their angles,
// once for all heads, into LDS; then a power of two of lanes takes a row (a
// token and a head of q, k or v), 8 elements a lane, so that the largest
// magnitude of a row to be quantised is a reduction over neighbouring lanes.
// With pairs (i, i + half) a lane reads its partner's 8 elements as well:
// they come from the caches, and no lane waits for another.
// An angle is the float64 product of the position and the frequency, brought
// to within an eighth turn there; in float32 a position of 10^5 would leave it
// 2^-8 off. Polynomials in float32 do the rest.
// Memory traffic bounds it: q, k and v are read once, q_out and the cells written
// once. Measured: 32767 tokens, 32 + 8 heads of 128, bf16 to e4m3, 741 MB: 155 us back to back, 4.8 TB/s,
// a large copy's rate; in a graph 163, 64 tokens 4.9 us, one 3.3. Rows a lane has in flight
// (2, 3, 4, 6): 177, 170, 178, 183 us; waves of queries alone leave out the largest magnitude
// and the scale: 160 us, 164 with them (before it). Offsets of 24-bit factors instead of 64: 8 % slower.
#include "extend.h"
#include "kdecode.h"

namespace convt {

namespace {

constexpr int kRows = 3;  // rows a lane has in flight

// Cosine and sine of a by their Taylor polynomials on |x| <= pi / 4, where the
// terms left out are below 2^-28; q counts quarter turns. Their number n is off
// by 2^-53 of itself, so an angle beyond some 2^50 is brought there in several
// steps (four for the largest there is). An infinite or NaN angle gives NaN.
__device__ __forceinline__ void turn(double a, float &c, float &s) {
    double r = a;
    int q = 0;
    do {
        const double n = rint(r * 0.63661977236758134308);
        r = fma(n, -1.5707963267948965580, r);
        r = fma(n, -6.1232339957367660359e-17, r);
        q += (int)(n - 4.0 * floor(n * 0.25));
    } while (fabs(r) > 0.79);
    const float x = (float)r, z = x * x;
    const float sp = x + x * z * (-1.0f / 6 + z * (1.0f / 120 + z * (-1.0f / 5040 + z * (1.0f / 362880))));
    const float cp = 1.0f + z * (-0.5f + z * (1.0f / 24 + z * (-1.0f / 720 + z * (1.0f / 40320 + z * (-1.0f / 3628800)))));
    const float ss = q & 1 ? cp : sp, cc = q & 1 ? sp : cp;
    s = q & 2 ? -ss : ss;
    c = (q + 1) & 2 ? -cc : cc;
}

// FULL: head_dim, rotary_dim and, with pairs (i, i + half), half are multiples
// of 8, so that a lane's 8 elements are of one kind. 1 << lanes_log2 lanes a row.
template <typename T, bool Q8, bool FULL>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a, int lanes_log2) {
    extern __shared__ float turns[];  // [block_tokens][half] cosines, then sines
    const CacheArgs &c = a.c;
    const int half = a.half, D = c.head_dim;
    float *cosines = turns, *sines = turns + a.block_tokens * half;
    const int per_token = a.heads + 2 * c.kv_heads;
    const int piece = (threadIdx.x & ((1 << lanes_log2) - 1)) * 8;
    const int group = threadIdx.x >> lanes_log2, groups = 256 >> lanes_log2;
    const int n = D - piece;  // elements of the lane's piece, 0 or less for none
    const int64_t step = (int64_t)gridDim.x * a.block_tokens;
    for (int64_t t0 = (int64_t)blockIdx.x * a.block_tokens; t0 < c.tokens; t0 += step) {
        const int tokens = c.tokens - t0 < a.block_tokens ? (int)(c.tokens - t0) : a.block_tokens;
        __syncthreads();
        for (int i = threadIdx.x; i < tokens * half; i += 256) {
            const int t = (int)fast_div((uint32_t)i, a.div_half);
            turn((double)a.positions[t0 + t] * (double)a.inv_freq[i - t * half], cosines[i], sines[i]);
        }
        __syncthreads();
        const int rows = tokens * per_token;
        // all lanes of a wave stay in the loop together, for the reduction
        for (int base = 0; base < rows; base += kRows * groups) {
            Raw8<T> raw[kRows], other[kRows];
            int64_t slot[kRows];
            int tok[kRows], head[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                // rows past the last read the last one and are not stored
                int row = base + u * groups + group;
                row = row < rows ? row : rows - 1;
                tok[u] = (int)fast_div((uint32_t)row, a.div_rows);
                head[u] = row - tok[u] * per_token;
                const int64_t t = t0 + tok[u];
                const T *src;
                if (head[u] < a.heads) src = (const T *)a.q + t * a.q_stride[0][0] + head[u] * a.q_stride[0][1];
                else if (head[u] < a.heads + c.kv_heads)
                    src = (const T *)c.k + t * c.row_stride[0][0] + (head[u] - a.heads) * c.row_stride[0][1];
                else src = (const T *)c.v + t * c.row_stride[1][0] + (head[u] - a.heads - c.kv_heads) * c.row_stride[1][1];
                slot[u] = c.slots[t];
                if constexpr (FULL) {
                    const int at = n > 0 ? piece : 0;
                    const bool turned = at < 2 * half && !a.interleaved;
                    raw[u] = load8<T>(src + at, 8);
                    other[u] = load8<T>(src + (turned ? (at < half ? at + half : at - half) : at), 8);
                } else {
                    raw[u] = n > 0 ? load8<T>(src + piece, n) : zero8<T>();
                    other[u] = zero8<T>();
                    if (!a.interleaved && n > 0) {
                        T *o = (T *)&other[u];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int d = piece + j;
                            if (j < n && d < 2 * half) o[j] = src[d < half ? d + half : d - half];
                        }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const bool real = base + u * groups + group < rows;
                const bool is_v = head[u] >= a.heads + c.kv_heads;
                float f[8], g[8];
                raw_to_f32<T>(raw[u], f);
                raw_to_f32<T>(other[u], g);
                if (!is_v && piece < 2 * half) {
                    const float *cs = cosines + tok[u] * half, *sn = sines + tok[u] * half;
                    float y[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int d = piece + j;
                        const bool second = a.interleaved ? j & 1 : d >= half;
                        const int i = a.interleaved ? d >> 1 : second ? d - half : d;
                        const float o = a.interleaved ? f[j ^ 1] : g[j];
                        if (FULL || d < 2 * half) y[j] = f[j] * cs[i] + (second ? o : -o) * sn[i];
                        else y[j] = f[j];
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = y[j];
                }
                if (head[u] < a.heads) {
                    if (real && n > 0)
                        store8<T>((T *)a.q_out + (t0 + tok[u]) * a.q_stride[1][0] + head[u] * a.q_stride[1][1] + piece, f, n);
                }
                if (!__any(head[u] >= a.heads)) continue;  // the wave's rows are all queries
                // the reduction is over all lanes, whatever their rows are
                float s = 1.0f;
                if constexpr (Q8) {
                    uint32_t amax[1] = {0};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t b = j < n ? abs_bits(f[j]) : 0;
                        amax[0] = b > amax[0] ? b : amax[0];
                    }
                    group_max_u32(amax, lanes_log2);
                    float inv;
                    s = row_scale(amax[0], inv);
                    for (int j = 0; j < 8; ++j) f[j] *= inv;
                }
                if (head[u] >= a.heads && real && n > 0) {
                    const Place p = place_of(c, slot[u]);
                    const int kvh = head[u] - a.heads - (is_v ? c.kv_heads : 0);
                    if (p.page >= 0) {
                        const int64_t at = cache_offset(c.cache_stride[is_v], kvh, p) + piece;
                        void *cells = is_v ? c.v_cache : c.k_cache;
                        if constexpr (Q8) {
                            store8_e4m3((uint8_t *)cells + at, f, n);
                            if (piece == 0) (is_v ? c.v_scale : c.k_scale)[scale_offset(c, kvh, p)] = s;
                        } else {
                            store8<T>((T *)cells + at, f, n);
                        }
                    }
                }
            }
        }
    }
}

template <typename T, bool Q8> void run(const AppendArgs &a, hipStream_t s) {
    int lanes_log2 = 0;
    while ((8 << lanes_log2) < a.c.head_dim) ++lanes_log2;
    const int64_t blocks = (a.c.tokens + a.block_tokens - 1) / a.block_tokens;
    const unsigned grid = (unsigned)(blocks < (1 << 20) ? blocks : (1 << 20));
    const size_t lds = (size_t)a.block_tokens * a.half * 2 * sizeof(float);
    const bool full = a.c.head_dim % 8 == 0 && a.half % (a.interleaved ? 4 : 8) == 0;
    if (full) append_kernel<T, Q8, true><<<grid, 256, lds, s>>>(a, lanes_log2);
    else append_kernel<T, Q8, false><<<grid, 256, lds, s>>>(a, lanes_log2);
}

}  // namespace

hipError_t launch_append(const AppendArgs &a, int dtype, int quantised, hipStream_t stream) {
    if (dtype == CONVT_DTYPE_F32) {
        if (quantised) run<float, true>(a, stream);
        else run<float, false>(a, stream);
    } else if (dtype == CONVT_DTYPE_BF16) {
        if (quantised) run<uint16_t, true>(a, stream);
        else run<uint16_t, false>(a, stream);
    } else {
        if (quantised) run<_Float16, true>(a, stream);
        else run<_Float16, false>(a, stream);
    }
    return hipGetLastError();
}

}  // namespace convt
