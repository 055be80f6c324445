// i8_gated_backward.hip -- gradients of the gated projection.
//
// With g, u the two scaled products (recomputed: the int32 sums are exact, so
// they are the forward pass's bits) and d the gradient of the output,
//     dg = d * u * act'(g),   du = d * act(g)
//     d_x[t][i]         = sum_f dg[t][f] gate_scale[f] w_gate[f][i] + du[t][f] up_scale[f] w_up[f][i]
//     d_gate_scale[f]   = sum_t dg[t][f] acc_gate[t][f] x_scale[t]
//     d_up_scale[f]     = sum_t du[t][f] acc_up[t][f] x_scale[t]
// d_x is the gradient with respect to the dequantised activation x * x_scale.
#include "ffn_common.hpp"

namespace loom {

namespace {

// One (token, channel) pair per thread: the two coefficients of d_x into
// coef[t][2 rows], and the 16 tokens' terms of the scale gradients into
// part[token tile][2 rows].
template <int TYPE>
__global__ __launch_bounds__(256) void coefficients_kernel(I8Product p, const void *d_out, int64_t d_stride,
                                                           float *__restrict__ coef, float *__restrict__ part) {
    typedef typename ElementOf<TYPE>::type T;
    __shared__ float terms[2][16][17];
    const int64_t tiles = (p.rows + 15) / 16;
    const int64_t n = (int64_t)(blockIdx.x % tiles) * 16 + (threadIdx.x & 15);
    const int64_t tile = blockIdx.x / tiles, t = tile * 16 + (threadIdx.x >> 4);
    float tg = 0.0f, tu = 0.0f;
    if (n < p.rows && t < p.tokens) {
        const int32_t *xr = p.x + t * p.kw, *wr = p.w + n * p.kw, *ur = p.w_up + n * p.kw;
        int acc = 0, up = 0;
        for (int j = 0; j < p.kw; ++j) {
            acc = __builtin_amdgcn_sdot4(wr[j], xr[j], acc, false);
            up = __builtin_amdgcn_sdot4(ur[j], xr[j], up, false);
        }
        const float xs = p.x_scale ? p.x_scale[t] : 1.0f;
        const float g = (float)acc * p.w_scale[n] * xs, u = (float)up * p.up_scale[n] * xs;
        const float d = (float)((const T *)d_out)[t * d_stride + n];
        float value, slope;
        act_value_slope(p.act, g, value, slope);
        const float dg = d * u * slope, du = d * value;
        coef[t * 2 * p.rows + n] = dg * p.w_scale[n];
        coef[t * 2 * p.rows + p.rows + n] = du * p.up_scale[n];
        tg = dg * ((float)acc * xs);
        tu = du * ((float)up * xs);
    }
    terms[0][threadIdx.x >> 4][threadIdx.x & 15] = tg;
    terms[1][threadIdx.x >> 4][threadIdx.x & 15] = tu;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int which = threadIdx.x >> 4, c = threadIdx.x & 15;
        const int64_t m = (int64_t)(blockIdx.x % tiles) * 16 + c;
        float sum = 0.0f;
        for (int i = 0; i < 16; ++i) sum = sum + terms[which][i][c];
        if (m < p.rows) part[tile * 2 * p.rows + which * (int64_t)p.rows + m] = sum;
    }
}

__global__ __launch_bounds__(256) void scale_gradients_kernel(const float *__restrict__ part, int64_t tiles,
                                                              int64_t rows, float *__restrict__ d_gate,
                                                              float *__restrict__ d_up) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= 2 * rows) return;
    float sum = 0.0f;
    for (int64_t i = 0; i < tiles; ++i) sum = sum + part[i * 2 * rows + c];
    float *to = c < rows ? d_gate : d_up;
    if (to) to[c < rows ? c : c - rows] = sum;
}

template <int TYPE>
__global__ __launch_bounds__(256) void d_x_kernel(I8Product p, const float *__restrict__ coef, void *d_x) {
    typedef typename ElementOf<TYPE>::type T;
    const int64_t k = 4 * (int64_t)p.kw, blocks = (k + 255) / 256;
    const int64_t i = (int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x, t = blockIdx.x / blocks;
    if (i >= k) return;
    const int8_t *wg = (const int8_t *)p.w, *wu = (const int8_t *)p.w_up;
    const float *c = coef + t * 2 * p.rows;
    float sum = 0.0f;
    for (int64_t f = 0; f < p.rows; ++f)
        sum = sum + c[f] * (float)wg[f * k + i] + c[p.rows + f] * (float)wu[f * k + i];
    ((T *)d_x)[t * k + i] = (T)sum;
}

template <int TYPE>
hipError_t run(const loom_launch_config &cfg, const I8Product &p, const void *d_out, int64_t d_stride, void *d_x,
               float *d_gate, float *d_up, void *workspace, hipStream_t stream) {
    float *coef = (float *)workspace, *part = coef + 2 * (int64_t)p.rows * p.tokens;
    const int64_t tiles = ((int64_t)p.tokens + 15) / 16;
    if (p.tokens > 0 && p.rows > 0)
        hipLaunchKernelGGL((coefficients_kernel<TYPE>), dim3(cfg.workgroups[0]), dim3(256), 0, stream, p, d_out,
                           d_stride, coef, part);
    if ((d_gate || d_up) && p.rows > 0)
        hipLaunchKernelGGL(scale_gradients_kernel, dim3((uint32_t)((2 * (int64_t)p.rows + 255) / 256)), dim3(256), 0,
                           stream, part, tiles, (int64_t)p.rows, d_gate, d_up);
    if (d_x && p.tokens > 0 && p.kw > 0)
        hipLaunchKernelGGL((d_x_kernel<TYPE>), dim3((uint32_t)(p.tokens * ((4 * (int64_t)p.kw + 255) / 256))),
                           dim3(256), 0, stream, p, coef, d_x);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_gated_projection_backward(const loom_launch_config &cfg, const I8Product &p, const void *d_out,
                                               int type, int64_t d_stride, void *d_x, float *d_gate, float *d_up,
                                               void *workspace, hipStream_t stream) {
    if (type == LOOM_F32)
        return run<LOOM_F32>(cfg, p, d_out, d_stride, d_x, d_gate, d_up, workspace, stream);
    if (type == LOOM_F16)
        return run<LOOM_F16>(cfg, p, d_out, d_stride, d_x, d_gate, d_up, workspace, stream);
    return run<LOOM_BF16>(cfg, p, d_out, d_stride, d_x, d_gate, d_up, workspace, stream);
}

}  // namespace loom
