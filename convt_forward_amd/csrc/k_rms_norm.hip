// Residual addition, root-mean-square norm and the optional e4m3 output.
//
//     h = x + residual;  y = h * (mean h^2 + eps)^(-1/2) * weight
//
// One pass over memory: a row's h stays in registers between the sum of
// squares, the largest |y| and the stores, so every input is read once and
// every output written once, which is what bounds the kernel (HBM). A row is
// held by LANES threads in NV pieces of 8 elements each: a wave for short
// rows (no barrier), a block of 256 for ordinary ones, of 1024 for long
// ones; rows longer than that are read a second time (norm_wide). All of a
// row's loads are in flight together, and 8 blocks a CU overlap one row's
// reductions with another's loads.
// Measured: 16384 rows x 8192, bf16 with residual to e4m3, 940 MB: 161 us, 5.8
// TB/s, the rate of a bare read; 77 rows x 5001, f16: 3.8 us a call of a graph;
// one row x 1024: 2.6, an empty launch (4.4 and 2.4 us in a kernel trace).
#include "decode.h"
#include "kdecode.h"

namespace convt {

namespace {

struct NormArgs {
    const void *x, *weight, *residual;
    void *y, *residual_out;
    float *scale;
    int64_t rows, x_stride, residual_stride, y_stride, residual_out_stride;
    int32_t width;
    float eps, inv_width;
};

// Sum (or largest) over the LANES threads that hold a row, given to all.
template <int LANES> __device__ __forceinline__ float row_sum(float v, float *lds) {
    v = wave_sum(v);
    if constexpr (LANES > 64) {
        const int wave = threadIdx.x / 64;
        __syncthreads();
        if (threadIdx.x % 64 == 0) lds[wave] = v;
        __syncthreads();
        v = 0.0f;
        for (int i = 0; i < LANES / 64; ++i) v += lds[i];
    }
    return v;
}
template <int LANES> __device__ __forceinline__ uint32_t row_max(uint32_t v, float *lds_f) {
    v = wave_max_u32(v);
    if constexpr (LANES > 64) {
        uint32_t *lds = (uint32_t *)lds_f;
        const int wave = threadIdx.x / 64;
        __syncthreads();
        if (threadIdx.x % 64 == 0) lds[wave] = v;
        __syncthreads();
        v = 0;
        for (int i = 0; i < LANES / 64; ++i) v = lds[i] > v ? lds[i] : v;
    }
    return v;
}

template <typename T, int LANES, int NV, bool Q>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void norm_kernel(NormArgs a) {
    constexpr int ROWS = LANES < 256 ? 256 / LANES : 1;  // rows of a block
    __shared__ float lds[16];
    const int lane = threadIdx.x % LANES;
    const T *weight = (const T *)a.weight;
    Raw8<T> w[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = (v * LANES + lane) * 8;
        w[v] = i < a.width ? load8<T>(weight + i, a.width - i) : zero8<T>();
    }
    // a block of several waves has one row, so its barriers are met by all
    for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; row < a.rows;
         row += (int64_t)gridDim.x * ROWS) {
        const T *x = (const T *)a.x + row * a.x_stride;
        Raw8<T> rx[NV], rr[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = (v * LANES + lane) * 8;
            rx[v] = i < a.width ? load8<T>(x + i, a.width - i) : zero8<T>();
        }
        if (a.residual) {
            const T *res = (const T *)a.residual + row * a.residual_stride;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int i = (v * LANES + lane) * 8;
                rr[v] = i < a.width ? load8<T>(res + i, a.width - i) : zero8<T>();
            }
        }
        float h[NV][8];
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) raw_to_f32<T>(rx[v], h[v]);
        if (a.residual) {
            T *out = (T *)a.residual_out + row * a.residual_out_stride;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int i = (v * LANES + lane) * 8;
                float f[8];
                raw_to_f32<T>(rr[v], f);
                for (int j = 0; j < 8; ++j) h[v][j] += f[j];
                if (i < a.width) store8<T>(out + i, h[v], a.width - i);
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            for (int j = 0; j < 8; ++j) sum += h[v][j] * h[v][j];
        const float rstd = 1.0f / sqrtf(row_sum<LANES>(sum, lds) * a.inv_width + a.eps);
        uint32_t amax = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float f[8];
            raw_to_f32<T>(w[v], f);
            for (int j = 0; j < 8; ++j) {
                h[v][j] = h[v][j] * rstd * f[j];
                if constexpr (Q) {
                    // places past the width hold 0, but NaN where rstd is infinite
                    const uint32_t b = (v * LANES + lane) * 8 + j < a.width ? abs_bits(h[v][j]) : 0;
                    amax = b > amax ? b : amax;
                }
            }
        }
        if constexpr (Q) {
            float inv;
            const float s = row_scale(row_max<LANES>(amax, lds), inv);
            uint8_t *y = (uint8_t *)a.y + row * a.y_stride;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int i = (v * LANES + lane) * 8;
                for (int j = 0; j < 8; ++j) h[v][j] *= inv;
                if (i < a.width) store8_e4m3(y + i, h[v], a.width - i);
            }
            if (lane == 0) a.scale[row] = s;
        } else {
            T *y = (T *)a.y + row * a.y_stride;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int i = (v * LANES + lane) * 8;
                if (i < a.width) store8<T>(y + i, h[v], a.width - i);
            }
        }
    }
}

// Rows too long for a block's registers: h is formed again in each pass (sum,
// largest, stores) from x and residual, whose second reading mostly meets the
// caches. residual_out may be residual or x, so it is written in the last
// pass, by the thread that has just read the same places.
template <typename T, bool Q>
__global__ __launch_bounds__(1024) void norm_wide(NormArgs a) {
    __shared__ float lds[16];
    const T *weight = (const T *)a.weight;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = (const T *)a.x + row * a.x_stride;
        const T *res = a.residual ? (const T *)a.residual + row * a.residual_stride : nullptr;
        auto load_h = [&](int i, float *h) {
            raw_to_f32<T>(load8<T>(x + i, a.width - i), h);
            if (res) {
                float f[8];
                raw_to_f32<T>(load8<T>(res + i, a.width - i), f);
                for (int j = 0; j < 8; ++j) h[j] += f[j];
            }
        };
        float sum = 0.0f;
        for (int i = threadIdx.x * 8; i < a.width; i += 1024 * 8) {
            float h[8];
            load_h(i, h);
            for (int j = 0; j < 8; ++j) sum += h[j] * h[j];
        }
        const float rstd = 1.0f / sqrtf(row_sum<1024>(sum, lds) * a.inv_width + a.eps);
        float inv = 1.0f;
        if constexpr (Q) {
            uint32_t amax = 0;
            for (int i = threadIdx.x * 8; i < a.width; i += 1024 * 8) {
                float h[8], f[8];
                load_h(i, h);
                raw_to_f32<T>(load8<T>(weight + i, a.width - i), f);
                for (int j = 0; j < 8; ++j) {
                    const uint32_t b = i + j < a.width ? abs_bits(h[j] * rstd * f[j]) : 0;
                    amax = b > amax ? b : amax;
                }
            }
            const float s = row_scale(row_max<1024>(amax, lds), inv);
            if (threadIdx.x == 0) a.scale[row] = s;
        }
        for (int i = threadIdx.x * 8; i < a.width; i += 1024 * 8) {
            float h[8], f[8];
            load_h(i, h);
            if (res) store8<T>((T *)a.residual_out + row * a.residual_out_stride + i, h, a.width - i);
            raw_to_f32<T>(load8<T>(weight + i, a.width - i), f);
            for (int j = 0; j < 8; ++j) h[j] = h[j] * rstd * f[j];
            if constexpr (Q) {
                for (int j = 0; j < 8; ++j) h[j] *= inv;
                store8_e4m3((uint8_t *)a.y + row * a.y_stride + i, h, a.width - i);
            } else {
                store8<T>((T *)a.y + row * a.y_stride + i, h, a.width - i);
            }
        }
    }
}

template <typename T, int LANES, int NV, bool Q> void run(const NormArgs &a, hipStream_t s) {
    constexpr int ROWS = LANES < 256 ? 256 / LANES : 1;
    const int64_t blocks = (a.rows + ROWS - 1) / ROWS;
    norm_kernel<T, LANES, NV, Q><<<(unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)), LANES < 256 ? 256 : LANES, 0, s>>>(a);
}

template <typename T, bool Q> void run_width(const NormArgs &a, hipStream_t s) {
    const int pieces = (a.width + 7) / 8;
    if (pieces <= 64) run<T, 64, 1, Q>(a, s);
    else if (pieces <= 128) run<T, 64, 2, Q>(a, s);
    else if (pieces <= 256) run<T, 256, 1, Q>(a, s);
    else if (pieces <= 512) run<T, 256, 2, Q>(a, s);
    else if (pieces <= 1024) run<T, 256, 4, Q>(a, s);
    else if (pieces <= 2048) run<T, 1024, 2, Q>(a, s);
    else if (pieces <= 4096) run<T, 1024, 4, Q>(a, s);
    else norm_wide<T, Q><<<(unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20)), 1024, 0, s>>>(a);
}

template <typename T> void run_type(const NormArgs &a, int quantise, hipStream_t s) {
    if (quantise) run_width<T, true>(a, s);
    else run_width<T, false>(a, s);
}

}  // namespace

hipError_t launch_rms_norm(const convt_rms_norm_problem &p, const void *x, const void *weight,
                           const void *residual, void *y, float *scale, void *residual_out,
                           hipStream_t stream) {
    NormArgs a{};
    a.x = x;
    a.weight = weight;
    a.residual = residual;
    a.y = y;
    a.residual_out = residual_out;
    a.scale = scale;
    a.rows = p.rows;
    // the stride of a single row is not read from the problem: row 0 is all
    a.x_stride = p.x_stride;
    a.residual_stride = p.residual_stride;
    a.y_stride = p.y_stride;
    a.residual_out_stride = p.residual_out_stride;
    a.width = (int32_t)p.width;
    a.eps = p.eps;
    a.inv_width = (float)(1.0 / (double)p.width);
    if (p.dtype == CONVT_DTYPE_F32) run_type<float>(a, p.quantise, stream);
    else if (p.dtype == CONVT_DTYPE_BF16) run_type<uint16_t>(a, p.quantise, stream);
    else run_type<_Float16>(a, p.quantise, stream);
    return hipGetLastError();
}

}  // namespace convt
