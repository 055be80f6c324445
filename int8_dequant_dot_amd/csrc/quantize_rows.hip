// quantize_rows.hip -- symmetric int8 quantisation of rows (tokens).
//
//     a = max |x[r][c]|,  scale[r] = a / 127,  q[r][c] = rint(x[r][c] * (127 / a))
//
// Both quotients are single f32 roundings, the product another, and rint
// rounds halves to even.  |x| <= a, so the product is at most 127 (1 + 2^-23)
// and q stays in [-127, 127].
#include "ffn_common.hpp"

namespace loom {

namespace {

template <int TYPE>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const typename ElementOf<TYPE>::type *__restrict__ x,
                                                            int rows, int64_t cols, int64_t row_stride,
                                                            int32_t *__restrict__ q, float *__restrict__ scale) {
    __shared__ float peaks[256];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const auto *src = x + row * row_stride;
        float top = 0.0f;
        bool finite = true;
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            const float v = (float)src[c];
            finite = finite && fabsf(v) <= 3.4028234663852886e38f;  // false for NaN
            top = fmaxf(top, fabsf(v));
        }
        peaks[threadIdx.x] = finite ? top : __builtin_inff();
        __syncthreads();
        for (int half = 128; half > 0; half >>= 1) {
            if ((int)threadIdx.x < half) peaks[threadIdx.x] = fmaxf(peaks[threadIdx.x], peaks[threadIdx.x + half]);
            __syncthreads();
        }
        top = peaks[0];
        __syncthreads();
        const bool ok = top <= 3.4028234663852886e38f, live = ok && top >= kQuantizeTiny;
        const float inverse = live ? 127.0f / top : 0.0f;
        if (threadIdx.x == 0) scale[row] = !ok ? __builtin_nanf("") : live ? top / 127.0f : 0.0f;
        for (int64_t j = threadIdx.x; j < cols / 4; j += 256) {
            uint32_t word = 0;
            for (int b = 0; b < 4; ++b) {
                const float v = (float)src[4 * j + b];
                const int i = live ? (int)rintf(v * inverse) : 0;
                word |= (uint32_t)(i & 0xFF) << (8 * b);
            }
            q[row * (cols / 4) + j] = (int32_t)word;
        }
    }
}

template <int TYPE>
void run(const loom_launch_config &cfg, const void *x, int rows, int64_t cols, int64_t row_stride, int32_t *q,
         float *scale, hipStream_t stream) {
    hipLaunchKernelGGL((quantize_rows_kernel<TYPE>), dim3(cfg.workgroups[0]), dim3(cfg.workgroup_size[0]), 0, stream,
                       (const typename ElementOf<TYPE>::type *)x, rows, cols, row_stride, q, scale);
}

}  // namespace

hipError_t launch_quantize_rows(const loom_launch_config &cfg, const void *x, int type, int rows, int64_t cols,
                                int64_t row_stride, int32_t *q, float *scale, hipStream_t stream) {
    if (type == LOOM_F32) run<LOOM_F32>(cfg, x, rows, cols, row_stride, q, scale, stream);
    else if (type == LOOM_F16) run<LOOM_F16>(cfg, x, rows, cols, row_stride, q, scale, stream);
    else run<LOOM_BF16>(cfg, x, rows, cols, row_stride, q, scale, stream);
    return hipGetLastError();
}

}  // namespace loom
