// i8_matmul.hip -- int8 matrix product with a scale for each token and each
// channel, and the gated projection (two products, the activation and the
// product of the two in one kernel).
//
//     acc[t][n] = sum_i w[n][i] * x[t][i]                       (exact, int32)
//     y[t][n]   = (f32(acc[t][n]) * w_scale[n]) * x_scale[t]    (two f32 roundings)
//     product:  out[t][n] = y[t][n] + bias[n]
//     gated:    out[t][n] = act(y_gate[t][n]) * y_up[t][n]
#include "ffn_common.hpp"

namespace loom {

namespace {

// One output per thread, 16 tokens x 16 channels per workgroup.
template <bool GATED, int TYPE>
__global__ __launch_bounds__(256) void i8_product_kernel(I8Product p) {
    typedef typename ElementOf<TYPE>::type T;
    const int64_t tiles = (p.rows + 15) / 16;
    const int64_t n = (int64_t)(blockIdx.x % tiles) * 16 + (threadIdx.x & 15);
    const int64_t t = (int64_t)(blockIdx.x / tiles) * 16 + (threadIdx.x >> 4);
    if (n >= p.rows || t >= p.tokens) return;
    const int32_t *xr = p.x + t * p.kw, *wr = p.w + n * p.kw, *ur = GATED ? p.w_up + n * p.kw : nullptr;
    int acc = 0, up = 0;
    for (int j = 0; j < p.kw; ++j) {
        acc = __builtin_amdgcn_sdot4(wr[j], xr[j], acc, false);
        if (GATED) up = __builtin_amdgcn_sdot4(ur[j], xr[j], up, false);
    }
    const float xs = p.x_scale ? p.x_scale[t] : 1.0f;
    float y = (float)acc * p.w_scale[n] * xs;
    if (GATED) y = act_value(p.act, y) * ((float)up * p.up_scale[n] * xs);
    else if (p.bias) y = y + p.bias[n];
    ((T *)p.out)[t * p.out_stride + n] = (T)y;
}

template <bool GATED>
hipError_t run(const loom_launch_config &cfg, const I8Product &p, int type, hipStream_t stream) {
    const dim3 grid(cfg.workgroups[0]), block(cfg.workgroup_size[0]);
    if (type == LOOM_F32) hipLaunchKernelGGL((i8_product_kernel<GATED, LOOM_F32>), grid, block, 0, stream, p);
    else if (type == LOOM_F16) hipLaunchKernelGGL((i8_product_kernel<GATED, LOOM_F16>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((i8_product_kernel<GATED, LOOM_BF16>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_matmul(const loom_launch_config &cfg, const I8Product &p, int type, hipStream_t stream) {
    return run<false>(cfg, p, type, stream);
}

hipError_t launch_i8_gated_projection(const loom_launch_config &cfg, const I8Product &p, int type,
                                      hipStream_t stream) {
    return run<true>(cfg, p, type, stream);
}

}  // namespace loom
