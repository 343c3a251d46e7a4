// Attention of one new token per stream over the paged cache: the direct
// kernel (any element type, head dimension, page size and alignment) and the
// joining of the length axis's parts. The matrix-core kernel is in
// k_attend_mfma.hip.
//
// The softmax runs on powers of two: with s = scale * log2(e) * <q, K[t]>,
// p[t] = 2^(s - m) over the running maximum m, l = sum p, O = sum p V, and a
// part (m, l, O) joins another after both are brought to the larger m.
#include "decode.h"
#include "kdecode.h"

namespace convt {

namespace {

constexpr int kWaves = 4;

// 64 tokens a wave and step. A lane first takes one token and the whole dot
// product with q (held in LDS), then the lanes turn to the head dimension and
// add the 64 values p[t] V[t], one token after the other. Simple and general;
// its loads of K run along the lanes' own rows, which the caches gather, and each
// query head reads its kv head again, so it stays well below the memory rate
// that the matrix-core kernel reaches (4 streams of 100-131 K, bf16: 3.1 ms against
// 0.33). It serves float32, odd head dimensions, pages and alignments.
template <typename T, bool Q8>
__global__ __launch_bounds__(64 * kWaves) void attend_direct(AttendArgs a) {
    typedef typename std::conditional<Q8, uint8_t, T>::type C;
    __shared__ float q_lds[kMaxHeadDim];
    __shared__ float o_lds[kWaves][kMaxHeadDim];
    __shared__ float m_lds[kWaves], l_lds[kWaves];
    const uint32_t b = fast_div(blockIdx.x, a.div_heads);
    const int h = (int)(blockIdx.x - b * (uint32_t)a.heads);
    const int kvh = h / a.share;
    const int chunk = blockIdx.y;
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    int len = a.lengths[b];
    len = len < 0 ? 0 : len > a.max_length ? a.max_length : len;
    const int t0 = chunk * a.chunk_tokens;
    if (t0 >= len && chunk > 0) return;  // the join knows how many parts there are
    const int t1 = len - t0 < a.chunk_tokens ? len : t0 + a.chunk_tokens;
    const int D = a.head_dim;

    const T *q = (const T *)a.q + b * a.q_stride[0] + h * a.q_stride[1];
    for (int d = threadIdx.x; d < D; d += 64 * kWaves) q_lds[d] = to_f32<T>(q[d]) * a.scale_log2e;
    __syncthreads();

    constexpr int NO = kMaxHeadDim / 64;
    float o[NO] = {};
    float m = -INFINITY, l = 0.0f;
    const int32_t *table = a.page_table + b * a.table_stride;
    for (int ts = t0 + wave * 64; ts < t1; ts += 64 * kWaves) {
        const int t = ts + lane;
        float s = -INFINITY, vs = 0.0f;
        int64_t voff = -1;  // the token's values, or -1 for one that is not seen
        if (t < t1) {
            const uint32_t pi = fast_div((uint32_t)t, a.div_page);
            const int64_t page = table[pi];
            if (page >= 0 && page < a.n_pages) {
                const int off = t - (int)pi * a.page_size;
                const C *k = (const C *)a.k_cache + page * a.k_stride[0] + kvh * a.k_stride[1] + off * a.k_stride[2];
                voff = page * a.v_stride[0] + kvh * a.v_stride[1] + off * a.v_stride[2];
                s = 0.0f;
                for (int d = 0; d < D; d += 8) {
                    float f[8];
                    if constexpr (Q8) e4m3_to_f32(load8_e4m3(k + d, D - d), f);
                    else raw_to_f32<T>(load8<T>(k + d, D - d), f);
                    for (int j = 0; j < 8; ++j)
                        if (d + j < D) s += f[j] * q_lds[d + j];
                }
                if constexpr (Q8) {
                    const int64_t si = (page * a.kv_heads + kvh) * a.page_size + off;
                    s *= a.k_scale[si];
                    vs = a.v_scale[si];
                }
            }
        }
        const float m_new = fmaxf(m, wave_max(s));
        // nothing seen yet (or scores of -infinity alone): any finite base
        const float base = m_new == -INFINITY ? 0.0f : m_new;
        const float alpha = exp2f(m - base);
        float p = voff >= 0 ? exp2f(s - base) : 0.0f;
        l = l * alpha + wave_sum(p);
        m = m_new;
        if constexpr (Q8) p *= vs;
#pragma unroll
        for (int i = 0; i < NO; ++i) o[i] *= alpha;
        for (uint64_t seen = __ballot(voff >= 0); seen; seen &= seen - 1) {
            const int j = __ffsll((unsigned long long)seen) - 1;
            const float pj = __shfl(p, j);
            const C *v = (const C *)a.v_cache + __shfl(voff, j);
#pragma unroll
            for (int i = 0; i < NO; ++i) {
                const int d = i * 64 + lane;
                if (d < D) {
                    float f;
                    if constexpr (Q8) f = __builtin_amdgcn_cvt_f32_fp8((int)v[d], 0);
                    else f = to_f32<T>(v[d]);
                    o[i] += pj * f;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NO; ++i) {
        const int d = i * 64 + lane;
        if (d < D) o_lds[wave][d] = o[i];
    }
    if (lane == 0) {
        m_lds[wave] = m;
        l_lds[wave] = l;
    }
    __syncthreads();
    float mm = -INFINITY;
    for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, m_lds[w]);
    const float base = mm == -INFINITY ? 0.0f : mm;
    float f[kWaves], ll = 0.0f;
    for (int w = 0; w < kWaves; ++w) {
        f[w] = exp2f(m_lds[w] - base);
        ll += l_lds[w] * f[w];
    }
    const int64_t part = ((int64_t)blockIdx.x * a.chunks + chunk);
    for (int d = threadIdx.x; d < D; d += 64 * kWaves) {
        float v = 0.0f;
        for (int w = 0; w < kWaves; ++w) v += o_lds[w][d] * f[w];
        if (a.chunks > 1) a.part_o[part * D + d] = v;
        else ((T *)a.out)[b * a.out_stride[0] + h * a.out_stride[1] + d] = from_f32<T>(ll == 0.0f ? 0.0f : v / ll);
    }
    if (threadIdx.x == 0) {
        if (a.chunks > 1) {
            a.part_ml[part * 2] = mm;
            a.part_ml[part * 2 + 1] = ll;
        } else if (a.lse) {
            a.lse[blockIdx.x] = (mm + log2f(ll)) * 0.69314718055994531f;
        }
    }
}

// Joins the parts of one (stream, head): out = sum 2^(m_c - m) O_c / sum
// 2^(m_c - m) l_c. 4 dims a thread, 1 << lanes_log2 threads a part, the
// block's other threads take other parts; blockIdx.y: the next dims, where
// there are so many parts that few dims a block (and more blocks) pay: 235
// parts of 16 heads of 256 dims take 4 us, 11 with all dims in one block.
template <typename T>
__global__ __launch_bounds__(256) void attend_join(AttendArgs a, int lanes_log2) {
    __shared__ float o_lds[256 * 4];
    __shared__ float m_lds[kWaves], l_lds[256];
    const uint32_t b = fast_div(blockIdx.x, a.div_heads);
    const int h = (int)(blockIdx.x - b * (uint32_t)a.heads);
    int len = a.lengths[b];
    len = len < 0 ? 0 : len > a.max_length ? a.max_length : len;
    // part 0 is there even for an empty stream (len + chunk_tokens may pass 31 bits)
    const int n = len > 0 ? (len - 1) / a.chunk_tokens + 1 : 1;
    const int D = a.head_dim;
    const int64_t part0 = (int64_t)blockIdx.x * a.chunks;
    const float *ml = a.part_ml + part0 * 2;
    float m = -INFINITY;
    for (int c = threadIdx.x; c < n; c += 256) m = fmaxf(m, ml[2 * c]);
    m = wave_max(m);
    if (threadIdx.x % 64 == 0) m_lds[threadIdx.x / 64] = m;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, m_lds[w]);
    const float base = m == -INFINITY ? 0.0f : m;
    const int lanes = 1 << lanes_log2, groups = 256 >> lanes_log2;
    const int d0 = blockIdx.y * 4 * lanes;
    const int d = d0 + (threadIdx.x & (lanes - 1)) * 4, group = threadIdx.x >> lanes_log2;
    f32x4 o = {0, 0, 0, 0};
    float l = 0.0f;
    if (d + 4 <= D) {
#pragma unroll 4
        for (int c = group; c < n; c += groups) {
            const float f = __builtin_amdgcn_exp2f(ml[2 * c] - base);
            l += ml[2 * c + 1] * f;
            o += f * *(const f32x4_a4 *)(a.part_o + (part0 + c) * D + d);
        }
    } else if (d < D) {
        for (int c = group; c < n; c += groups) {
            const float f = __builtin_amdgcn_exp2f(ml[2 * c] - base);
            l += ml[2 * c + 1] * f;
            for (int j = 0; j < 3; ++j)
                if (d + j < D) o[j] += f * a.part_o[(part0 + c) * D + d + j];
        }
    }
    for (int j = 0; j < 4; ++j) o_lds[threadIdx.x * 4 + j] = o[j];
    l_lds[threadIdx.x] = l;
    __syncthreads();
    l = 0.0f;
    for (int g = 0; g < groups; ++g) l += l_lds[g << lanes_log2];  // the lanes of a part agree
    for (int i = threadIdx.x; i < 4 * lanes && d0 + i < D; i += 256) {
        float v = 0.0f;
        for (int g = 0; g < groups; ++g) v += o_lds[(g << lanes_log2) * 4 + i];
        ((T *)a.out)[b * a.out_stride[0] + h * a.out_stride[1] + d0 + i] = from_f32<T>(l == 0.0f ? 0.0f : v / l);
    }
    if (threadIdx.x == 0 && blockIdx.y == 0 && a.lse) a.lse[blockIdx.x] = (m + log2f(l)) * 0.69314718055994531f;
}

template <typename T> void run_direct(const AttendArgs &a, int quantised, hipStream_t s) {
    const dim3 grid((unsigned)a.batch * (unsigned)a.heads, (unsigned)a.chunks);
    if (quantised) attend_direct<T, true><<<grid, 64 * kWaves, 0, s>>>(a);
    else attend_direct<T, false><<<grid, 64 * kWaves, 0, s>>>(a);
}

}  // namespace

hipError_t launch_attend_direct(const AttendArgs &a, int dtype, int quantised, hipStream_t stream) {
    if (dtype == CONVT_DTYPE_F32) run_direct<float>(a, quantised, stream);
    else if (dtype == CONVT_DTYPE_BF16) run_direct<uint16_t>(a, quantised, stream);
    else run_direct<_Float16>(a, quantised, stream);
    return hipGetLastError();
}

hipError_t launch_attend_join(const AttendArgs &a, int dtype, hipStream_t stream) {
    int lanes_log2 = 0;
    while ((4 << lanes_log2) < a.head_dim) ++lanes_log2;
    // at least 32 dims, 128 bytes, of a part
    while (lanes_log2 > 3 && a.chunks > 4 * (256 >> lanes_log2)) --lanes_log2;
    const dim3 grid((unsigned)a.batch * (unsigned)a.heads, (unsigned)((a.head_dim + (4 << lanes_log2) - 1) / (4 << lanes_log2)));
    if (dtype == CONVT_DTYPE_F32) attend_join<float><<<grid, 256, 0, stream>>>(a, lanes_log2);
    else if (dtype == CONVT_DTYPE_BF16) attend_join<uint16_t><<<grid, 256, 0, stream>>>(a, lanes_log2);
    else attend_join<_Float16><<<grid, 256, 0, stream>>>(a, lanes_log2);
    return hipGetLastError();
}

}  // namespace convt
