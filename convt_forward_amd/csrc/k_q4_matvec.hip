// Products of a few rows with 4-bit weights and group scales: the direct
// kernel (any element type, any group that is a multiple of 8, any alignment).
// The matrix-core kernel is in k_q4_mfma.hip.
#include "decode.h"
#include "kdecode.h"

namespace convt {

namespace {

struct Q4Args {
    const void *x, *w, *scales;
    const float *x_scale;
    void *y;
    int64_t x_stride, y_stride;
    int32_t rows, n, k, group;
};

constexpr int kRows = 8;  // rows of x a wave carries at once

// A wave per output column n: each lane takes 8 consecutive k at a time, its
// 8 weights in one word, and up to 8 rows of x against them. The group's
// scale multiplies the lane's sum of 8 products, all in float32. Unpacking and
// multiplying bound it (16 e4m3 rows x 8192 x 32768: 497 us against 34 on the
// matrix cores); it serves float32 and what those do not take.
template <typename T, bool X8>
__global__ __launch_bounds__(256) void q4_direct(Q4Args a) {
    typedef typename std::conditional<X8, uint8_t, T>::type X;
    const int lane = threadIdx.x % 64;
    const int64_t n = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (n >= a.n) return;
    const uint8_t *w = (const uint8_t *)a.w + n * (a.k / 2);
    const T *sc = (const T *)a.scales + n * (a.k / a.group);
    for (int64_t m0 = (int64_t)blockIdx.y * kRows; m0 < a.rows; m0 += (int64_t)gridDim.y * kRows) {
        const int mr = a.rows - m0 < kRows ? (int)(a.rows - m0) : kRows;
        float acc[kRows] = {};
        for (int64_t k = lane * 8; k < a.k; k += 512) {
            const uint32_t word = *(const u32_a1 *)(w + k / 2);
            const float s = to_f32<T>(sc[k / a.group]);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = (float)((int)(word >> (4 * j) & 15u) - 8);
#pragma unroll
            for (int m = 0; m < kRows; ++m) {
                if (m < mr) {
                    const X *x = (const X *)a.x + (m0 + m) * a.x_stride + k;
                    float xf[8];
                    if constexpr (X8) e4m3_to_f32(load8_e4m3(x, 8), xf);
                    else raw_to_f32<T>(load8<T>(x, 8), xf);
                    float v = 0.0f;
                    for (int j = 0; j < 8; ++j) v += f[j] * xf[j];
                    acc[m] += v * s;
                }
            }
        }
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
            const float v = wave_sum(acc[m]);
            if (m < mr && lane == 0)
                ((T *)a.y)[(m0 + m) * a.y_stride + n] = from_f32<T>(X8 ? v * a.x_scale[m0 + m] : v);
        }
    }
}

template <typename T> void run(const Q4Args &a, int x8, hipStream_t s) {
    const int64_t my = (a.rows + kRows - 1) / kRows;
    const dim3 grid((unsigned)((a.n + 3) / 4), (unsigned)(my < 4096 ? my : 4096));
    if (x8) q4_direct<T, true><<<grid, 256, 0, s>>>(a);
    else q4_direct<T, false><<<grid, 256, 0, s>>>(a);
}

}  // namespace

hipError_t launch_q4_direct(const convt_q4_problem &p, const void *x, const float *x_scale, const void *w,
                            const void *scales, void *y, hipStream_t stream) {
    const Q4Args a{x, w, scales, x_scale, y, p.x_stride, p.y_stride, (int32_t)p.rows, (int32_t)p.n, (int32_t)p.k,
                   (int32_t)p.group};
    if (p.dtype == CONVT_DTYPE_F32) run<float>(a, p.x_quantised, stream);
    else if (p.dtype == CONVT_DTYPE_BF16) run<uint16_t>(a, p.x_quantised, stream);
    else run<_Float16>(a, p.x_quantised, stream);
    return hipGetLastError();
}

}  // namespace convt
