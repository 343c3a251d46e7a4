// Attention of one new token per stream over the paged cache, on the matrix
// cores: two-byte element types, caches of that type or of e4m3 codes.
//
// Reading the keys and values bounds it (HBM), so the layout serves the loads:
// every wave streams its own 32-token steps straight into registers in the
// operand layout of v_mfma_f32_16x16x32, with no LDS and no barrier until the
// block's waves are joined. The rows of a tile are the (up to 16) query heads
// that share a kv head, so a key is read once for all of them.
//
//   scores   S^T = K Q^T: A is 16 tokens x 32 dims of K as stored (lane: token
//            lane % 16, 8 consecutive dims), B is Q. A score tile then has the
//            head in lane % 16 and 4 tokens a lane, so a head's maximum is
//            over the lane's own values and two lane swaps.
//   values   O^T += V^T P^T: B wants, for its lane's head, 8 tokens: exactly
//            the 4 + 4 scores the lane already holds of the step's two tiles
//            (the sum over tokens may run in any order as long as A agrees).
//            A wants 8 tokens of one dim; a lane loads the same VD = DP / 16
//            dims of its 8 tokens with wide loads and transposes them in
//            registers, one v_perm_b32 for two elements.
//
// K of the next step is requested once the scores are formed, V of the next
// step once O is updated, each into the registers just freed.
//
// Roundings: Q and K enter as stored (e4m3 codes are exact in bf16 and f16;
// their scales multiply the float32 scores). p (times the value's scale) is
// rounded to float16 where V is float16: 2^-11 of its value. For that it carries
// a factor 2^15 (p <= 1, so 2^15 p fits, and float16's steps are relative from
// 2^-14 on), which the waves' join takes off: weights down to 2^-29 of the
// wave's largest keep their 11 bits, and smaller ones are off by at most 2^-40
// of it. Where V is bfloat16 or e4m3, p goes in as the sum of two bfloat16
// values (2^-16), since one bfloat16 (2^-8) would be as coarse as the output
// itself; the second product costs nothing beside the loads. Its V has the
// largest finite value where V is infinite: the low part may be 0 or negative,
// and the first product carries the infinity.
//
// Measured (kernel alone, then with the join): 4 streams of 100-131 K tokens, 8 kv
// heads of 128, bf16, 1.89 GB: 327, 333 us, 5.8 TB/s; 32 ragged streams up to
// 4096, e4m3, 139 MB: 34, 39 us, 4.1 TB/s. Of these some 5 us do not shrink
// with the bytes (launch, the loads from a length to a page to its keys, the
// join); the products and conversions are hidden (leaving them out: the
// same time). 2 or 8 waves a block: 42, 47 us on the ragged batch; loads marked
// as not to be kept: 2 % faster beyond the 256 MB cache, 15 % slower inside it.
#include "decode.h"
#include "kdecode.h"

namespace convt {

namespace {

constexpr int kWaves = 4;
constexpr int kStep = 32;  // tokens a wave takes at a time

// Over the four lanes that share lane % 16.
__device__ __forceinline__ float quad_max(float v) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int BYTES> struct Piece;
template <> struct Piece<4> { typedef uint32_t type; };
template <> struct Piece<8> { typedef u32x2 type; };
template <> struct Piece<16> { typedef u32x4 type; };

// E: type of q, out and of an unquantised cache. DP: head_dim rounded up to 64,
// 128 or 256. FULL: head_dim == DP. The second launch bound is the blocks of
// a CU that the registers are held to: 4, 3 and 1 by DP.
template <typename E, bool Q8, int DP, bool FULL>
__global__ __launch_bounds__(64 * kWaves, DP == 64 ? 4 : DP == 128 ? 3 : 1) void attend_mfma(AttendArgs a, int head_tiles) {
    typedef typename std::conditional<Q8, __bf16, E>::type EV;  // P and V
    typedef typename Vec8<E>::type E8;
    typedef typename Vec8<EV>::type EV8;
    constexpr bool SPLIT = __is_same(EV, __bf16);
    constexpr float RAISE = SPLIT ? 1.0f : 0x1p15f;  // the factor that p and o carry
    constexpr int CS = Q8 ? 1 : 2;        // bytes of a cache element
    constexpr int NC = DP / 32;           // products of 32 dims for a score tile
    constexpr int KL = Q8 ? DP / 64 : NC; // 16-byte loads of a lane for a score tile
    constexpr int VD = DP / 16;           // dims of V a lane holds
    constexpr int VW = VD * CS / 4;       // words of them for one token
    constexpr int VP = VW > 4 ? 16 : VW * 4;  // bytes of one load
    constexpr int VL = VW * 4 / VP;           // loads of a token
    constexpr int LD = DP + 4;            // spacing of the heads' sums in LDS
    __shared__ float o_lds[kWaves][16 * LD];
    __shared__ float m_lds[kWaves][16], l_lds[kWaves][16];

    const int lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int ht = blockIdx.x % head_tiles;
    const int kvh = blockIdx.x / head_tiles % a.kv_heads;
    const int b = blockIdx.x / head_tiles / a.kv_heads;
    const int head0 = kvh * a.share + ht * 16;
    const int nheads = a.share - ht * 16 < 16 ? a.share - ht * 16 : 16;
    const int chunk = blockIdx.y;
    int len = a.lengths[b];
    len = len < 0 ? 0 : len > a.max_length ? a.max_length : len;
    const int t0 = chunk * a.chunk_tokens;
    if (t0 >= len && chunk > 0) return;  // the join knows how many parts there are
    const int t1 = len - t0 < a.chunk_tokens ? len : t0 + a.chunk_tokens;
    const int D = FULL ? DP : a.head_dim;

    // Q as the B operand of each product; dims in the order K's loads have.
    E8 q[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int d = Q8 ? (c / 2) * 64 + g * 16 + (c % 2) * 8 : c * 32 + g * 8;
        u32x4 w = {0, 0, 0, 0};
        if (r < nheads && (FULL || d < D))
            w = *(const u32x4 *)((const uint16_t *)a.q + b * a.q_stride[0] + (head0 + r) * a.q_stride[1] + d);
        q[c] = __builtin_bit_cast(E8, w);
    }

    // byte offsets of the lane inside a tile of 16 tokens
    const char *kc = (const char *)a.k_cache, *vc = (const char *)a.v_cache;
    const int64_t k_lane = (r * a.k_stride[2] + g * (16 / CS)) * CS;
    const int v_dim = FULL || r * VD < D ? r * VD : 0;  // lanes past D read dim 0 and are not stored
    const int64_t v_lane = (g * 4 * a.v_stride[2] + v_dim) * CS;
    const int32_t *table = a.page_table + b * a.table_stride;

    u32x4 kr[2][KL];
    typename Piece<VP>::type vr[8][VL];
    f32x4 ks[2] = {}, vs[2] = {};
    bool ok[2];
    int64_t page[2];
    int off[2];

    // The pages of the two tiles of a step. A tile past the end takes the
    // last one there is; its tokens are masked by their index.
    int32_t entry[2];
    int entry_off[2];
    auto look_up = [&](int ts) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            int t = ts + 16 * u;
            const int last = (t1 - 1) & ~15;
            t = t < last ? t : last;
            const int pi = (int)fast_div((uint32_t)t, a.div_page);
            entry[u] = table[pi];
            entry_off[u] = t - pi * a.page_size;
        }
    };
    auto take_entries = [&]() {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            ok[u] = entry[u] >= 0 && entry[u] < a.n_pages;
            page[u] = ok[u] ? entry[u] : 0;
            off[u] = entry_off[u];
        }
    };
    auto load_k = [&]() {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const char *base = kc + (page[u] * a.k_stride[0] + kvh * a.k_stride[1] + off[u] * a.k_stride[2]) * CS + k_lane;
#pragma unroll
            for (int c = 0; c < KL; ++c) {
                if constexpr (FULL) {
                    kr[u][c] = *(const u32x4 *)(base + c * 64);
                } else {
                    // dims past D: nothing is read, and K is 0 there as Q is
                    const int d = c * (64 / CS) + g * (16 / CS);
                    kr[u][c] = d < D ? *(const u32x4 *)(base + c * 64) : u32x4{0, 0, 0, 0};
                }
            }
        }
    };
    auto load_v = [&]() {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const char *base = vc + (page[u] * a.v_stride[0] + kvh * a.v_stride[1] + off[u] * a.v_stride[2]) * CS + v_lane;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < VL; ++i)
                    vr[u * 4 + j][i] = *(const typename Piece<VP>::type *)(base + j * a.v_stride[2] * CS + i * VP);
        }
    };
    auto load_scales = [&]() {
        if constexpr (Q8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t at = (page[u] * a.kv_heads + kvh) * a.page_size + off[u] + g * 4;
                ks[u] = *(const f32x4 *)(a.k_scale + at);
                vs[u] = *(const f32x4 *)(a.v_scale + at);
            }
        }
    };

    f32x4 o[VD];
#pragma unroll
    for (int j = 0; j < VD; ++j) o[j] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    int ts = t0 + wave * kStep;
    if (ts < t1) {
        look_up(ts);
        take_entries();
        load_scales();
        load_k();
        load_v();
    }
    // The next step's loads are issued without a condition (past the end they
    // read the last tile again, from the caches): the compiler's waits count
    // the loads in flight on the path with the fewest, so a branch around
    // them would make every wait one for all.
    for (; ts < t1; ts += kWaves * kStep) {
        const int next = ts + kWaves * kStep;
        const bool partial = ts + kStep > t1 || !ok[0] || !ok[1];
        const bool seen0 = ok[0], seen1 = ok[1];
        look_up(next);
        f32x4 s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            s[u] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                u32x4 w;
                if constexpr (Q8) {
                    const uint32_t w0 = kr[u][c / 2][(c % 2) * 2], w1 = kr[u][c / 2][(c % 2) * 2 + 1];
                    w = u32x4{e4m3_pair<E, false>(w0), e4m3_pair<E, true>(w0), e4m3_pair<E, false>(w1),
                              e4m3_pair<E, true>(w1)};
                } else {
                    w = kr[u][c];
                }
                s[u] = mfma16(__builtin_bit_cast(E8, w), q[c], s[u]);
            }
        }
        // The phases of a step stay apart: mixed, their temporaries would not
        // fit in the registers of the waves a SIMD should hold.
        __builtin_amdgcn_sched_barrier(0);
        f32x4 vscale[2] = {vs[0], vs[1]};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            s[u] *= a.scale_log2e;
            if constexpr (Q8) s[u] *= ks[u];
        }
        take_entries();
        load_scales();
        load_k();
        __builtin_amdgcn_sched_barrier(0);
        if (partial) {
            // unseen tokens: no weight, and their values (whatever they
            // hold) become 0
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool seen = (u ? seen1 : seen0) && ts + u * 16 + g * 4 + i < t1;
                    s[u][i] = seen ? s[u][i] : -INFINITY;
                    vscale[u][i] = seen ? vscale[u][i] : 0.0f;
#pragma unroll
                    for (int k = 0; k < VL; ++k)
                        vr[u * 4 + i][k] = seen ? vr[u * 4 + i][k] : typename Piece<VP>::type{};
                }
        }
        float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                          fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        top = fmaxf(m, quad_max(top));
        // scores of -infinity alone so far: any finite base
        const float base = top == -INFINITY ? 0.0f : top;
        if (__any(top != m)) {
            const float alpha = __builtin_amdgcn_exp2f(m - base);
            l *= alpha;
#pragma unroll
            for (int j = 0; j < VD; ++j) o[j] *= alpha;
            m = top;
        }
        float p[8];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = __builtin_amdgcn_exp2f(s[u][i] - base);
                l += e;
                p[u * 4 + i] = Q8 ? e * vscale[u][i] : e * RAISE;
            }
        u32x4 ph, pl;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ph[i] = pack_half2<EV>(p[2 * i], p[2 * i + 1]);
            if constexpr (SPLIT)
                pl[i] = pack_half2<EV>(p[2 * i] - __uint_as_float(ph[i] << 16),
                                       p[2 * i + 1] - __uint_as_float(ph[i] & 0xffff0000u));
        }
        // V^T: two dims (one word of each token) at a time
#pragma unroll
        for (int jw = 0; jw < VD / 2; ++jw) {
            __builtin_amdgcn_sched_barrier(0);
            uint32_t w[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if constexpr (Q8) {
                    const int at = jw / 2;
                    uint32_t x;
                    if constexpr (VW == 1) x = vr[t][0];
                    else x = vr[t][0][at];
                    w[t] = jw % 2 ? e4m3_pair<EV, true>(x) : e4m3_pair<EV, false>(x);
                } else {
                    w[t] = vr[t][jw * 4 / VP][jw % (VP / 4)];
                }
            }
            u32x4 lo = {lo_pair(w[0], w[1]), lo_pair(w[2], w[3]), lo_pair(w[4], w[5]), lo_pair(w[6], w[7])};
            u32x4 hi = {hi_pair(w[0], w[1]), hi_pair(w[2], w[3]), hi_pair(w[4], w[5]), hi_pair(w[6], w[7])};
            o[2 * jw] = mfma16(__builtin_bit_cast(EV8, lo), __builtin_bit_cast(EV8, ph), o[2 * jw]);
            o[2 * jw + 1] = mfma16(__builtin_bit_cast(EV8, hi), __builtin_bit_cast(EV8, ph), o[2 * jw + 1]);
            if constexpr (SPLIT) {
                if constexpr (!Q8)  // e4m3 has no infinities
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        lo[i] = finite_bf16(lo[i]);
                        hi[i] = finite_bf16(hi[i]);
                    }
                o[2 * jw] = mfma16(__builtin_bit_cast(EV8, lo), __builtin_bit_cast(EV8, pl), o[2 * jw]);
                o[2 * jw + 1] = mfma16(__builtin_bit_cast(EV8, hi), __builtin_bit_cast(EV8, pl), o[2 * jw + 1]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        load_v();
    }

    // Join the waves: lane (head r, rows 4g + i) holds dims VD (4g + i) + j.
    l = quad_sum(l);
    if (r < nheads) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < VD; ++j) o_lds[wave][r * LD + VD * (4 * g + i) + j] = o[j][i];
        if (g == 0) {
            m_lds[wave][r] = m;
            l_lds[wave][r] = l;
        }
    }
    __syncthreads();
    for (int h = threadIdx.x / 64; h < nheads; h += kWaves) {
        float mm = -INFINITY;
        for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, m_lds[w][h]);
        const float base = mm == -INFINITY ? 0.0f : mm;
        float f[kWaves], ll = 0.0f;
        for (int w = 0; w < kWaves; ++w) {
            f[w] = __builtin_amdgcn_exp2f(m_lds[w][h] - base);
            ll += l_lds[w][h] * f[w];
        }
        const int64_t row = (int64_t)b * a.heads + head0 + h;
        const int64_t part = row * a.chunks + chunk;
        for (int d = lane; d < D; d += 64) {
            float v = 0.0f;
            for (int w = 0; w < kWaves; ++w) v += o_lds[w][h * LD + d] * f[w];
            v *= 1.0f / RAISE;
            if (a.chunks > 1)
                a.part_o[part * D + d] = v;
            else
                ((uint16_t *)a.out)[b * a.out_stride[0] + (head0 + h) * a.out_stride[1] + d] =
                    f32_to_half<E>(ll == 0.0f ? 0.0f : v / ll);
        }
        if (lane == 0) {
            if (a.chunks > 1) {
                a.part_ml[part * 2] = mm;
                a.part_ml[part * 2 + 1] = ll;
            } else if (a.lse) {
                a.lse[row] = (mm + log2f(ll)) * 0.69314718055994531f;
            }
        }
    }
}

template <typename E, bool Q8> void run(const AttendArgs &a, hipStream_t s) {
    const int head_tiles = (a.share + 15) / 16;
    const dim3 grid((unsigned)a.batch * a.kv_heads * head_tiles, (unsigned)a.chunks);
    const int D = a.head_dim;
    if (D == 64) attend_mfma<E, Q8, 64, true><<<grid, 64 * kWaves, 0, s>>>(a, head_tiles);
    else if (D < 64) attend_mfma<E, Q8, 64, false><<<grid, 64 * kWaves, 0, s>>>(a, head_tiles);
    else if (D == 128) attend_mfma<E, Q8, 128, true><<<grid, 64 * kWaves, 0, s>>>(a, head_tiles);
    else if (D < 128) attend_mfma<E, Q8, 128, false><<<grid, 64 * kWaves, 0, s>>>(a, head_tiles);
    else if (D == 256) attend_mfma<E, Q8, 256, true><<<grid, 64 * kWaves, 0, s>>>(a, head_tiles);
    else attend_mfma<E, Q8, 256, false><<<grid, 64 * kWaves, 0, s>>>(a, head_tiles);
}

}  // namespace

hipError_t launch_attend_mfma(const AttendArgs &a, int dtype, int quantised, hipStream_t stream) {
    if (dtype == CONVT_DTYPE_BF16) {
        if (quantised) run<__bf16, true>(a, stream);
        else run<__bf16, false>(a, stream);
    } else {
        if (quantised) run<_Float16, true>(a, stream);
        else run<_Float16, false>(a, stream);
    }
    return hipGetLastError();
}

}  // namespace convt
