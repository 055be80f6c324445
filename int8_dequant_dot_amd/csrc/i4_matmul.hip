// i4_matmul.hip -- products of int8 activations with 4-bit weights that have a
// scale for each channel and group of k; dense, or over routes grouped by expert,
// there also gated.
//
//     y[t][n]  = (sum_g scale[n][g] * f32(sum_{i in g} q[n][i] x[t][i])) * x_scale[t]
//     product: out[t][n] = y[t][n] + bias[n],   gated: act(y_gate) * y_up
//
// A group's sum is exact in int32; the groups are added in f32.
#include "i4_tiles.hpp"

namespace loom {

namespace {

// One wave a block of 32 tokens x 32 channels (gated: of both projections).
// A operand: 32 tokens, B: 32 channels; lane l holds 16 elements of k, from
// 16 (l >> 5) on, of token or channel l & 31, and of the sums channel l & 31,
// tokens 8 (r >> 2) + 4 (l >> 5) + (r & 3).
template <bool ROUTED, bool GATED, int ST>
__global__ __launch_bounds__(kI4Waves * kWave) void i4_block_kernel(I4Product p, int type) {
    const int lane = lane_id(), wave = threadIdx.x / kWave, half = lane >> 5;
    const int64_t blocks = (p.rows + 32 * kI4Waves - 1) / (32 * kI4Waves);
    const int64_t tile = blockIdx.x / blocks, n0 = (blockIdx.x % blocks) * (32 * kI4Waves) + wave * 32;
    int expert = 0, rows;
    int64_t t0;
    if constexpr (ROUTED) {
        if (!routed_tile<32>(p, tile, expert, t0, rows)) return;
    } else {
        t0 = tile * 32;
        rows = (int)min((int64_t)32, p.tokens - t0);
    }
    if (n0 >= p.rows) return;
    const int64_t n = min(n0 + (lane & 31), (int64_t)p.rows - 1), t = t0 + min(lane & 31, rows - 1);
    int64_t xr = t;
    float xs = 1.0f;
    if constexpr (ROUTED) {
        if (!x_row(p, t, xr)) xs = __builtin_nanf("");
    }
    if (p.x_scale) xs *= p.x_scale[xr];
    const int64_t wr = (int64_t)expert * p.rows + n;
    const int4v *x = (const int4v *)p.x + xr * p.chunks * 2 + half;
    const int4v *w = (const int4v *)p.w + wr * p.chunks, *u = GATED ? (const int4v *)p.w_up + wr * p.chunks : w;
    float acc[GATED ? 2 : 1][16];
#pragma unroll
    for (int m = 0; m < (GATED ? 2 : 1); ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[m][r] = 0.0f;
    const int per = 1 << p.chunk_shift;  // 32-element chunks of a group
    for (int g = 0; g < p.groups; ++g) {
        int16v sum[2] = {};
        for (int c = g * per; c < min(g * per + per, p.chunks); ++c) {
            const int4v a = x[2 * c];
#pragma unroll
            for (int m = 0; m < (GATED ? 2 : 1); ++m) {
                const int4v v = m ? u[c] : w[c];
                sum[m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, half ? i4_high(v) : i4_low(v), sum[m], 0, 0, 0);
            }
        }
#pragma unroll
        for (int m = 0; m < (GATED ? 2 : 1); ++m) {
            const float s = scale_at<ST>(m ? p.up_scale : p.w_scale, wr * p.groups + g);
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[m][r] = __builtin_fmaf((float)sum[m][r], s, acc[m][r]);
        }
    }
    const bool there = n0 + (lane & 31) < p.rows;
    const float bias = !GATED && p.bias ? p.bias[wr] : 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int row = 8 * (r >> 2) + 4 * half + (r & 3);
        const float scale = __shfl(xs, row);
        float y = acc[0][r] * kI4Unit * scale;
        if constexpr (GATED) y = act_value(p.act, y) * (acc[GATED ? 1 : 0][r] * kI4Unit * scale);
        else if (p.bias) y = y + bias;
        if (there && row < rows) store1(p.out, type, (t0 + row) * p.out_stride + n, y);
    }
}

template <bool ROUTED, typename C, int ST>
__global__ __launch_bounds__(C::NW * kWave, 1) void i4_tile_kernel(I4Product p, int type) {
    __shared__ __align__(1024) char lds[C::kLds];
    const uint32_t ch_tiles = count_of(p.rows, C::OUT_CH);
    I4TileLoop<C, ST> loop{p, lds};
    loop.lane = lane_id(), loop.half = loop.lane >> 5, loop.m = loop.lane & 31;
    loop.wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    loop.wm = loop.wave % C::WM, loop.wn = loop.wave / C::WM;
    loop.expert = 0;
    uint32_t ch, tok;
    if constexpr (ROUTED) {
        tile_of(blockIdx.x, ch_tiles, gridDim.x / ch_tiles, 1, ch, tok);
        if (!routed_tile<C::TK>(p, tok, loop.expert, loop.t0, loop.rows)) return;
    } else {
        tile_of(blockIdx.x, ch_tiles, count_of(p.tokens, C::TK), 8, ch, tok);
        loop.t0 = (int64_t)tok * C::TK;
        loop.rows = (int)min((int64_t)C::TK, p.tokens - loop.t0);
    }
    loop.n0 = (int64_t)ch * C::OUT_CH;
    loop.run([&](int r) {
        int64_t row = loop.t0 + r;
        if constexpr (ROUTED) x_row(p, loop.t0 + r, row);
        return row;
    });
    loop.store(type, [&](int r) {
        int64_t row = loop.t0 + r;
        float scale = 1.0f;
        if constexpr (ROUTED)
            if (!x_row(p, loop.t0 + r, row)) scale = __builtin_nanf("");
        return p.x_scale ? scale * p.x_scale[row] : scale;
    });
}

template <bool ROUTED, bool GATED, int ST>
hipError_t run(const loom_launch_config &cfg, const I4Product &p, int type, hipStream_t stream) {
    const dim3 grid(cfg.workgroups[0]), block(cfg.workgroup_size[0]);
    const int subs = i4_subs(p.chunk_shift);
    if (i4_use_tiles(p.tokens, ROUTED ? p.experts : 0)) {
        if (subs == 1) hipLaunchKernelGGL((i4_tile_kernel<ROUTED, I4Tile<2, 2, 1, GATED>, ST>), grid, block, 0, stream, p, type);
        else if (subs == 2) hipLaunchKernelGGL((i4_tile_kernel<ROUTED, I4Tile<2, 2, 2, GATED>, ST>), grid, block, 0, stream, p, type);
        else hipLaunchKernelGGL((i4_tile_kernel<ROUTED, I4Tile<2, 2, 4, GATED>, ST>), grid, block, 0, stream, p, type);
    } else {
        hipLaunchKernelGGL((i4_block_kernel<ROUTED, GATED, ST>), grid, block, 0, stream, p, type);
    }
    return hipGetLastError();
}

template <bool ROUTED, bool GATED>
hipError_t run_typed(const loom_launch_config &cfg, const I4Product &p, int scale_type, int type, hipStream_t stream) {
    switch (scale_type) {
        case LOOM_F32: return run<ROUTED, GATED, LOOM_F32>(cfg, p, type, stream);
        case LOOM_F16: return run<ROUTED, GATED, LOOM_F16>(cfg, p, type, stream);
        default: return run<ROUTED, GATED, LOOM_BF16>(cfg, p, type, stream);
    }
}

}  // namespace

hipError_t launch_i4_product(const loom_launch_config &cfg, const I4Product &p, I4Form form, int scale_type, int type,
                             hipStream_t stream) {
    if (form == kI4Dense) return run_typed<false, false>(cfg, p, scale_type, type, stream);
    if (form == kI4Routed) return run_typed<true, false>(cfg, p, scale_type, type, stream);
    return run_typed<true, true>(cfg, p, scale_type, type, stream);
}

}  // namespace loom
