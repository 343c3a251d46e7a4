// Attention of several new tokens per stream over the paged cache: the
// direct kernel (any element type, head dimension, page size and alignment)
// and the joining of the length axis's parts. The matrix-core kernel is in
// kextend_mfma.h, its instances in k_extend_{bf16,f16}{,_q8}.hip.
//
// The softmax runs on powers of two: with s = scale * log2(e) * <q, K[t]>,
// p[t] = 2^(s - m) over the running maximum m, l = sum p, O = sum p V, and a
// part (m, l, O) joins another after both are brought to the larger m.
#include "extend.h"
#include "kdecode.h"
#include "kextend.h"

namespace convt {

namespace {

constexpr int kWaves = 4;

// One block for a row (token and query head) and a part of what it sees. 64
// tokens a wave and step: a lane first takes one token and the whole dot product
// with q (held in LDS), then the lanes turn to the head dimension and add the
// 64 values p[t] V[t], one token after the other; a token that the row does not
// see is not read. Simple and general: every row reads its keys again, so it
// is far from the matrix-core kernel (a prompt of 8192 in a window of 4096: 100 ms
// against 0.45; one token of 64 streams: 1.9 ms against 0.10). It serves float32, odd head
// dimensions, pages and alignments.
template <typename T, bool Q8, bool TREE>
__global__ __launch_bounds__(64 * kWaves) void extend_direct(ExtendArgs a) {
    typedef typename std::conditional<Q8, uint8_t, T>::type C;
    __shared__ float q_lds[kMaxHeadDim];
    __shared__ float o_lds[kWaves][kMaxHeadDim];
    __shared__ float m_lds[kWaves], l_lds[kWaves];
    const int token = (int)fast_div(blockIdx.x, a.div_heads);
    const int h = (int)(blockIdx.x - (uint32_t)token * (uint32_t)a.heads);
    const int kvh = h / a.share;
    const int chunk = blockIdx.y;
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int D = a.head_dim;

    // What the row sees: v counts `first` first tokens, then those from lo on.
    int b, len, first = 0, lo = 0, n;
    const uint64_t *bits = nullptr;
    int64_t q_at, out_at;
    if constexpr (TREE) {
        b = (int)fast_div((uint32_t)token, a.div_drafts);
        const int i = token - b * a.drafts;
        len = cut_length(a, b);
        n = len + a.drafts < a.max_length ? len + a.drafts : a.max_length;
        bits = a.tree + b * a.tree_stride[0] + i * a.tree_stride[1];
        q_at = b * a.q_stride[0] + i * a.q_stride[1];
        out_at = b * a.out_stride[0] + i * a.out_stride[1];
    } else {
        int end;
        b = stream_of(a, token, end);
        if (b < 0) return;  // a row of no stream
        len = cut_length(a, b);
        const int pos = len - (end - token);
        lo = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
        first = a.sinks < lo ? a.sinks : lo;
        n = pos < 0 ? 0 : first + (pos - lo + 1);
        q_at = token * a.q_stride[1];
        out_at = token * a.out_stride[1];
    }
    const int64_t part = (int64_t)blockIdx.x * a.chunks + chunk;
    const int v0 = chunk * a.chunk_tokens;
    if (a.chunks > 1 && chunk == 0 && threadIdx.x == 0) a.part_count[blockIdx.x] = n > 0 ? (n - 1) / a.chunk_tokens + 1 : 1;
    if (v0 >= n && chunk > 0) return;  // the join knows how many parts there are
    const int v1 = n - v0 < a.chunk_tokens ? n : v0 + a.chunk_tokens;

    const T *q = (const T *)a.q + q_at + h * a.q_stride[2];
    for (int d = threadIdx.x; d < D; d += 64 * kWaves) q_lds[d] = to_f32<T>(q[d]) * a.scale_log2e;
    __syncthreads();

    constexpr int NO = kMaxHeadDim / 64;
    float o[NO] = {};
    float m = -INFINITY, l = 0.0f;
    const int32_t *table = a.page_table + b * a.table_stride;
    for (int vs0 = v0 + wave * 64; vs0 < v1; vs0 += 64 * kWaves) {
        const int v = vs0 + lane;
        const int t = v < first ? v : v - first + lo;
        float s = -INFINITY, vs = 0.0f;
        int64_t voff = -1;  // the token's values, or -1 for one that is not seen
        bool seen = v < v1;
        if constexpr (TREE)
            if (seen && t >= len) seen = bits[(t - len) >> 6] >> ((t - len) & 63) & 1;
        if (seen) {
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
        for (uint64_t left = __ballot(voff >= 0); left; left &= left - 1) {
            const int j = __ffsll((unsigned long long)left) - 1;
            const float pj = __shfl(p, j);
            const C *vr = (const C *)a.v_cache + __shfl(voff, j);
#pragma unroll
            for (int i = 0; i < NO; ++i) {
                const int d = i * 64 + lane;
                if (d < D) {
                    float f;
                    if constexpr (Q8) f = __builtin_amdgcn_cvt_f32_fp8((int)vr[d], 0);
                    else f = to_f32<T>(vr[d]);
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
    for (int d = threadIdx.x; d < D; d += 64 * kWaves) {
        float v = 0.0f;
        for (int w = 0; w < kWaves; ++w) v += o_lds[w][d] * f[w];
        if (a.chunks > 1) a.part_o[part * D + d] = v;
        else ((T *)a.out)[out_at + h * a.out_stride[2] + d] = from_f32<T>(ll == 0.0f ? 0.0f : v / ll);
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

// Joins the parts of a row: out = sum 2^(m_c - m) O_c / sum 2^(m_c - m) l_c. A
// part that saw nothing (m = -infinity, l = 0) has no O. 256 / ROWS threads a
// row: 1 << lanes_log2 of them take 4 dims each, the others other parts.
// ROWS = 1 where there are more than 16 parts, 4 where there are fewer. Reading the parts bounds it: 65536
// rows of 128 dims, up to 3 parts: 21 us; 4096 rows, up to 18: 11 us. Attention and join, us, ROWS = 1 and 4: 32 rows of
// up to 32 parts: 13.9, 16.0; 1024 of 52: 35, 42; 96 of 21: 22, 26; 192 of 21: 28.5, 30; 512 of 7: 17.9, 18.2; 1024 of 10: 21.5, 20.2;
// 3200 of 16: 53.9, 52.7; 12800 of 11: 62.5, 53.0; 16384 of 12: 107, 95; but 16384 of 32: 178, 174.
template <typename T, int ROWS>
__global__ __launch_bounds__(256) void extend_join(ExtendArgs a, int lanes_log2) {
    constexpr int PER = 256 / ROWS;
    __shared__ float o_lds[256 * 4];
    __shared__ float m_lds[4], l_lds[256];
    const int sub = threadIdx.x / PER, tid = threadIdx.x % PER;
    const uint32_t rows = (uint32_t)a.tokens * (uint32_t)a.heads;
    const uint32_t at = blockIdx.x * ROWS + sub;
    const uint32_t row = at < rows ? at : rows - 1;
    const int token = (int)fast_div(row, a.div_heads);
    const int h = (int)(row - (uint32_t)token * (uint32_t)a.heads);
    bool real = at < rows;
    int64_t out_at;
    if (a.tree) {
        const int b = (int)fast_div((uint32_t)token, a.div_drafts);
        out_at = b * a.out_stride[0] + (token - b * a.drafts) * a.out_stride[1];
    } else {
        real = real && (!a.starts || (token >= a.starts[0] && token < a.starts[a.batch]));
        out_at = token * a.out_stride[1];
    }
    // (rows that decreasing starts left to no block have any count)
    const int D = a.head_dim, count = real ? a.part_count[row] : 0, n = count < a.chunks ? count : a.chunks;
    real = n > 0;
    const float *ml = a.part_ml + (int64_t)row * a.chunks * 2;
    float m = -INFINITY;
    for (int c = tid; c < n; c += PER) m = fmaxf(m, ml[2 * c]);
    m = wave_max(m);
    if constexpr (ROWS == 1) {
        if (tid % 64 == 0) m_lds[tid / 64] = m;
        __syncthreads();
        for (int w = 0; w < 4; ++w) m = fmaxf(m, m_lds[w]);
    }
    const float base = m == -INFINITY ? 0.0f : m;
    const int lanes = 1 << lanes_log2, groups = PER >> lanes_log2;
    const int lane = tid & (lanes - 1), group = tid >> lanes_log2;
    // 4 * lanes dims at a time (head_dim up to 512 with 64 lanes takes two turns)
    for (int d0 = 0; d0 < D; d0 += 4 * lanes) {
        const int d = d0 + lane * 4;
        f32x4 o = {0, 0, 0, 0};
        float l = 0.0f;
#pragma unroll 4
        for (int c = group; c < n; c += groups) {
            const float mc = ml[2 * c], lc = ml[2 * c + 1];
            if (mc == -INFINITY && lc == 0.0f) continue;
            const float f = __builtin_amdgcn_exp2f(mc - base);
            l += lc * f;
            const float *po = a.part_o + ((int64_t)row * a.chunks + c) * D + d;
            if (d + 4 <= D) {
                o += f * *(const f32x4_a4 *)po;
            } else {
                for (int j = 0; j < 3; ++j)
                    if (d + j < D) o[j] += f * po[j];
            }
        }
        __syncthreads();
        for (int j = 0; j < 4; ++j) o_lds[threadIdx.x * 4 + j] = o[j];
        l_lds[threadIdx.x] = l;
        __syncthreads();
        l = 0.0f;
        for (int g = 0; g < groups; ++g) l += l_lds[sub * PER + (g << lanes_log2)];  // the lanes of a part agree
        for (int i = tid; i < 4 * lanes && d0 + i < D; i += PER) {
            float v = 0.0f;
            for (int g = 0; g < groups; ++g) v += o_lds[(sub * PER + (g << lanes_log2)) * 4 + i];
            if (real) ((T *)a.out)[out_at + h * a.out_stride[2] + d0 + i] = from_f32<T>(l == 0.0f ? 0.0f : v / l);
        }
        if (d0 == 0 && tid == 0 && real && a.lse) a.lse[row] = (m + log2f(l)) * 0.69314718055994531f;
    }
}

template <typename T> void run_direct(const ExtendArgs &a, int quantised, hipStream_t s) {
    const dim3 grid((unsigned)a.tokens * (unsigned)a.heads, (unsigned)a.chunks);
    if (a.tree) {
        if (quantised) extend_direct<T, true, true><<<grid, 64 * kWaves, 0, s>>>(a);
        else extend_direct<T, false, true><<<grid, 64 * kWaves, 0, s>>>(a);
    } else {
        if (quantised) extend_direct<T, true, false><<<grid, 64 * kWaves, 0, s>>>(a);
        else extend_direct<T, false, false><<<grid, 64 * kWaves, 0, s>>>(a);
    }
}

template <typename T> void run_join(const ExtendArgs &a, hipStream_t s) {
    int lanes_log2 = 0;
    while (lanes_log2 < 6 && (4 << lanes_log2) < a.head_dim) ++lanes_log2;
    const unsigned rows = (unsigned)a.tokens * (unsigned)a.heads;
    if (a.chunks > 16) extend_join<T, 1><<<rows, 256, 0, s>>>(a, lanes_log2);
    else extend_join<T, 4><<<(rows + 3) / 4, 256, 0, s>>>(a, lanes_log2);
}

}  // namespace

hipError_t launch_extend_direct(const ExtendArgs &a, int dtype, int quantised, hipStream_t stream) {
    if (dtype == CONVT_DTYPE_F32) run_direct<float>(a, quantised, stream);
    else if (dtype == CONVT_DTYPE_BF16) run_direct<uint16_t>(a, quantised, stream);
    else run_direct<_Float16>(a, quantised, stream);
    return hipGetLastError();
}

hipError_t launch_extend_join(const ExtendArgs &a, int dtype, hipStream_t stream) {
    if (dtype == CONVT_DTYPE_F32) run_join<float>(a, stream);
    else if (dtype == CONVT_DTYPE_BF16) run_join<uint16_t>(a, stream);
    else run_join<_Float16>(a, stream);
    return hipGetLastError();
}

}  // namespace convt
