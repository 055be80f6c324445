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

// Few tokens: the weights stream once from memory, straight into the matrix cores'
// operand registers.  A workgroup owns 32 weight rows (gated: 16 gate rows and the
// same 16 up rows); its waves each take a contiguous share of k in records of 32 rows
// x 256 bytes (512 elements), and their partial sums are added in wave order.  One
// load reads 4 rows x 256 contiguous bytes: lane l holds bytes 64 (l & 3) +
// 16 (l >> 4) .. + 15 of row 4 i + (l >> 2 & 3), so a product's 16 rows are 4 weight
// rows x 4 segments of 128 elements, and the 16 columns of B are 4 token slots x the
// same segments.  Of the sums only those of equal segments are wanted: element
// e = l & 3 of lane l, row 4 i + (l >> 4), slot 4 v + (l >> 2 & 3); they are scaled and
// added in f32.
//
// A segment of 128 is a group, or a part of one.  Of shorter groups it holds SUB = 2 or
// 4: a token then takes SUB slots, each of which sees the quarters l >> 4 of its own
// group and zeros elsewhere.
//
// Memory bounds it: one token x 16384 x 8192 in groups of 128 takes 13.1 us (5.3 TB/s, of
// it about 2.4 us a launch), the gated rows of 32 tokens x 8 routes over 128 experts of
// 2048 x 4096 168 to 171 us (6.5 to 6.6 TB/s).  A workgroup of 16 rows took 14.8 and 250 us, three
// records in flight 16.7 and 310, eight waves 18.7 and 257; 64-bit addresses instead of
// offsets from the tile 13.7 and 222.
template <int ST, int RI, int VG>
struct I4Record {
    int4v w[RI], x[VG][2];
    typename ElementOf<ST>::type scale[RI];
};

template <bool ROUTED, bool GATED, int ST, int VG>
__global__ __launch_bounds__(kWave * kI4StreamWaves, 2) void i4_stream_kernel(I4Product p, int type) {
    constexpr int KS = kI4StreamWaves, RI = kI4StreamLoads, ROWS = 4 * RI, OC = GATED ? ROWS / 2 : ROWS, kSlots = 4 * VG;
    __shared__ float part[KS][kSlots * ROWS];
    const int lane = lane_id(), m = lane & 15, quarter = lane >> 4, slot = m >> 2, segment = m & 3;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int sub_shift = 2 - min(p.chunk_shift, 2), sub = slot & ((1 << sub_shift) - 1), fit = kSlots >> sub_shift;
    const uint32_t blocks = count_of(p.rows, OC);
    int expert = 0, tokens = p.tokens;
    int64_t t0 = 0;
    uint32_t block = blockIdx.x;
    if constexpr (ROUTED) {
        const uint32_t tile = blockIdx.x / blocks;
        block = blockIdx.x - tile * blocks;
        if (!routed_tile(p, fit, tile, expert, t0, tokens)) return;
    }
    const int64_t n0 = (int64_t)block * OC, row0 = (int64_t)expert * p.rows + n0;
    const int left = (int)min((int64_t)OC, p.rows - n0);
    const int at = 4 * segment + quarter;  // 32-element chunk of the record
    // offsets from the tile's first rows, whose addresses are the same in every lane
    typedef typename ElementOf<ST>::type Scale;
    const int4v *const wbase[2] = {(const int4v *)p.w + row0 * p.chunks, (const int4v *)(GATED ? p.w_up : p.w) + row0 * p.chunks};
    const Scale *const sbase[2] = {(const Scale *)p.w_scale + row0 * p.groups,
                                   (const Scale *)(GATED ? p.up_scale : p.w_scale) + row0 * p.groups};
    const int4v *xrow[VG];
    uint32_t wrow[RI], srow[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        // row 4 i + slot of the operand, 4 i + quarter of the sums
        wrow[i] = (uint32_t)(min((4 * i + slot) % OC, left - 1) * p.chunks + at);
        srow[i] = (uint32_t)(min((4 * i + quarter) % OC, left - 1) * p.groups);
    }
    bool live[VG];
#pragma unroll
    for (int v = 0; v < VG; ++v) {
        const int token = (4 * v + slot) >> sub_shift;
        live[v] = token < tokens && quarter >> (2 - sub_shift) == sub;
        int64_t row = t0 + min(token, tokens - 1);
        if constexpr (ROUTED) x_row(p, row, row);
        xrow[v] = (const int4v *)p.x + row * p.chunks * 2 + 2 * at;
    }
    float acc[RI][VG];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int v = 0; v < VG; ++v) acc[i][v] = 0.0f;
    auto consume = [&](const I4Record<ST, RI, VG> &q) {
        int4v b[VG][2];
#pragma unroll
        for (int v = 0; v < VG; ++v) {
            b[v][0] = live[v] ? q.x[v][0] : int4v{};
            b[v][1] = live[v] ? q.x[v][1] : int4v{};
        }
        // two rows of products at a time: more would cost registers, and with them waves
#pragma unroll
        for (int i0 = 0; i0 < RI; i0 += 2) {
            int4v d[2][VG];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int4v low = i4_low(q.w[i0 + i]);
#pragma unroll
                for (int v = 0; v < VG; ++v) d[i][v] = __builtin_amdgcn_mfma_i32_16x16x64_i8(low, b[v][0], int4v{}, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int4v high = i4_high(q.w[i0 + i]);
#pragma unroll
                for (int v = 0; v < VG; ++v) d[i][v] = __builtin_amdgcn_mfma_i32_16x16x64_i8(high, b[v][1], d[i][v], 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int v = 0; v < VG; ++v) {
                    const int4v e = d[i][v];
                    const int lo = segment & 1 ? e[1] : e[0], hi = segment & 1 ? e[3] : e[2];
                    acc[i0 + i][v] = __builtin_fmaf((float)(segment & 2 ? hi : lo), (float)q.scale[i0 + i], acc[i0 + i][v]);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const int all = p.chunks / 16, per_wave = (all + KS - 1) / KS;
    const int first = min(all, wave * per_wave), records = min(all, first + per_wave) - first;
    int c = first * 16;
    const int group_at = 4 * segment + (sub << (2 - sub_shift));
    pipelined<2, I4Record<ST, RI, VG>>(
        records,
        [&]() {
            I4Record<ST, RI, VG> q;
#pragma unroll
            for (int i = 0; i < RI; ++i) q.w[i] = __builtin_nontemporal_load(wbase[i >= RI / 2] + wrow[i] + (uint32_t)c);
#pragma unroll
            for (int i = 0; i < RI; ++i) q.scale[i] = sbase[i >= RI / 2][srow[i] + (uint32_t)((c + group_at) >> p.chunk_shift)];
#pragma unroll
            for (int v = 0; v < VG; ++v) q.x[v][0] = xrow[v][2 * c], q.x[v][1] = xrow[v][2 * c + 1];
            c += 16;
            return q;
        },
        consume);
    if (p.chunks % 16 && wave == KS - 1) {  // the rest of the row: chunks past it are zero
        const bool there = all * 16 + at < p.chunks, grouped = all * 16 + group_at < p.chunks;
        I4Record<ST, RI, VG> q;
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            q.w[i] = there ? wbase[i >= RI / 2][wrow[i] + (uint32_t)(all * 16)] : int4v{};
            // no group, no scale: a sum of 0 stays 0 whatever the last group's scale is (read all the same: eight
            // branches around the loads cost 1.3 of 18 us at 1 x 16384 x 8224)
            const Scale scale = sbase[i >= RI / 2][srow[i] + (uint32_t)min((all * 16 + group_at) >> p.chunk_shift, p.groups - 1)];
            q.scale[i] = grouped ? scale : (Scale)0.0f;
        }
#pragma unroll
        for (int v = 0; v < VG; ++v) {
            q.x[v][0] = there ? xrow[v][2 * all * 16] : int4v{};
            q.x[v][1] = there ? xrow[v][2 * all * 16 + 1] : int4v{};
        }
        consume(q);
    }
    // each quad adds its output's 4 segments; its first lane publishes the sum
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int v = 0; v < VG; ++v) {
            const float t = group_sum<2>(acc[i][v]);
            if (segment == 0) part[wave][(4 * v + slot) * ROWS + 4 * i + quarter] = t;
        }
    __syncthreads();
    for (int o = threadIdx.x; o < fit * OC; o += kWave * KS) {
        const int t = o / OC, r = o % OC;
        if (t >= tokens || r >= left) continue;
        float sum = 0.0f, up = 0.0f;
#pragma unroll
        for (int w = 0; w < KS; ++w)
            for (int u = 0; u < 1 << sub_shift; ++u) {
                const float *from = &part[w][((t << sub_shift) + u) * ROWS + r];
                sum += from[0];
                if (GATED) up += from[OC];
            }
        int64_t row = t0 + t;
        float xs = 1.0f;
        if constexpr (ROUTED)
            if (!x_row(p, row, row)) xs = __builtin_nanf("");
        if (p.x_scale) xs *= p.x_scale[row];
        float y = sum * kI4Unit * xs;
        if (GATED) y = act_value(p.act, y) * (up * kI4Unit * xs);
        else if (p.bias) y = y + p.bias[row0 + r];
        store1(p.out, type, (t0 + t) * p.out_stride + n0 + r, y);
    }
}

// Two waves a SIMD are asked for where the shape has them: the compiler then leaves the
// products' sums in vector registers, where they are converted (5 to 8 % of a tile of four
// waves).  Several split waves (of one wave's tile each) share a tile: each takes a run of k over
// LDS of its own, with no barrier, and the sums are added in their order at the end.
template <bool ROUTED, typename C, int ST>
__global__ __launch_bounds__(C::kShape.waves() * kWave, C::kShape.waves() >= 4 ? 2 : 1) void i4_tile_kernel(I4Product p, int type) {
    constexpr int S = C::kShape.split;
    static_assert(S == 1 || (C::NW == 1 && C::kLds >= C::XT * C::WT * 4096), "the sums fit the steps");
    __shared__ __align__(1024) char lds[S * C::kLds];
    const uint32_t ch_tiles = count_of(p.rows, C::OUT_CH);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    I4TileLoop<C, ST> loop{p, lds + (S > 1 ? wave * C::kLds : 0)};
    loop.lane = lane_id(), loop.half = loop.lane >> 5, loop.m = loop.lane & 31;
    loop.wave = S > 1 ? 0 : wave;
    loop.wm = loop.wave % C::WM, loop.wn = loop.wave / C::WM;
    loop.expert = 0;
    uint32_t ch, tok;
    if constexpr (ROUTED) {
        tile_of(blockIdx.x, ch_tiles, gridDim.x / ch_tiles, 1, ch, tok);
        if (!routed_tile(p, C::TK, tok, loop.expert, loop.t0, loop.rows)) return;
    } else {
        tile_of(blockIdx.x, ch_tiles, count_of(p.tokens, C::TK), 8, ch, tok);
        loop.t0 = (int64_t)tok * C::TK;
        loop.rows = (int)min((int64_t)C::TK, p.tokens - loop.t0);
    }
    loop.n0 = (int64_t)ch * C::OUT_CH;
    const int all = p.chunks / (4 * C::PARTS), begin = S > 1 ? (int)((int64_t)all * wave / S) : 0;
    const int end = S > 1 ? (int)((int64_t)all * (wave + 1) / S) : all;
    loop.run(begin, end - begin, S == 1 || wave == S - 1, [&](int r) {
        int64_t row = loop.t0 + r;
        if constexpr (ROUTED) x_row(p, loop.t0 + r, row);
        return row;
    });
    auto scale_of = [&](int r) {
        int64_t row = loop.t0 + r;
        float scale = 1.0f;
        if constexpr (ROUTED)
            if (!x_row(p, loop.t0 + r, row)) scale = __builtin_nanf("");
        return p.x_scale ? scale * p.x_scale[row] : scale;
    };
    if constexpr (S > 1) {
        constexpr int N = 16 / S;  // sums of each block that a wave adds and stores
#pragma unroll
        for (int x = 0; x < C::XT; ++x)
#pragma unroll
            for (int w = 0; w < C::WT; ++w)
#pragma unroll
                for (int r = 0; r < 16; ++r) ((float *)loop.lds)[((x * C::WT + w) * 16 + r) * kWave + loop.lane] = loop.acc[x][w][r];
        __syncthreads();
#pragma unroll
        for (int x = 0; x < C::XT; ++x)
#pragma unroll
            for (int w = 0; w < C::WT; ++w)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    float sum = 0.0f;
#pragma unroll
                    for (int q = 0; q < S; ++q)
                        sum += ((const float *)(lds + q * C::kLds))[((x * C::WT + w) * 16 + wave * N + e) * kWave + loop.lane];
                    loop.acc[x][w][e] = sum;
                }
        loop.template store<N>(type, wave * N, scale_of);
    } else {
        loop.template store<16>(type, 0, scale_of);
    }
}

template <bool ROUTED, bool GATED, int ST, int SHAPE = 0>
void launch_tile(int shape, int subs, dim3 grid, dim3 block, const I4Product &p, int type, hipStream_t stream) {
    if constexpr (SHAPE < kI4TileCount) {
        if (shape != SHAPE) return launch_tile<ROUTED, GATED, ST, SHAPE + 1>(shape, subs, grid, block, p, type, stream);
        if (subs == 1) hipLaunchKernelGGL((i4_tile_kernel<ROUTED, I4Tile<SHAPE, 1, GATED>, ST>), grid, block, 0, stream, p, type);
        else if (subs == 2) hipLaunchKernelGGL((i4_tile_kernel<ROUTED, I4Tile<SHAPE, 2, GATED>, ST>), grid, block, 0, stream, p, type);
        else hipLaunchKernelGGL((i4_tile_kernel<ROUTED, I4Tile<SHAPE, 4, GATED>, ST>), grid, block, 0, stream, p, type);
    }
}

template <bool ROUTED, bool GATED, int ST>
hipError_t run(const loom_launch_config &cfg, const I4Product &p, int type, hipStream_t stream) {
    const dim3 grid(cfg.workgroups[0]), block(cfg.workgroup_size[0]);
    const int64_t experts = ROUTED ? p.experts : 0;
    const int subs = i4_subs(p.chunk_shift), slots = i4_stream_slots(p.tokens, experts, subs);
    if (slots == 4) {
        hipLaunchKernelGGL((i4_stream_kernel<ROUTED, GATED, ST, 1>), grid, block, 0, stream, p, type);
    } else if (slots == 8) {  // dense only
        if constexpr (!ROUTED) hipLaunchKernelGGL((i4_stream_kernel<false, false, ST, 2>), grid, block, 0, stream, p, type);
    } else {
        launch_tile<ROUTED, GATED, ST>(i4_tile_choice(p.rows, 32 * (int64_t)p.chunks, p.tokens, experts, GATED, subs), subs, grid,
                                       block, p, type, stream);
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
