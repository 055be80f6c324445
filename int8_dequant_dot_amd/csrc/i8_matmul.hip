// i8_matmul.hip -- int8 matrix product with a scale for each token and each
// channel, and the gated projection (two products, the activation and the
// product of the two in one kernel).
//
//     acc[t][n] = sum_i w[n][i] * x[t][i]                       (exact, int32)
//     y[t][n]   = (f32(acc[t][n]) * w_scale[n]) * x_scale[t]    (two f32 roundings)
//     product:  out[t][n] = y[t][n] + bias[n]
//     gated:    out[t][n] = act(y_gate[t][n]) * y_up[t][n]
#include "i8_tiles.hpp"

namespace loom {

namespace {

// Up to 16 tokens: the weights stream once from memory, straight into the matrix
// cores' operand registers.  A workgroup owns 16 weight rows (gated: 8 gate rows
// and the same 8 up rows); its KS waves each take a contiguous share of k in
// records of 16 rows x 256 bytes, and their int32 partial sums are added in wave
// order.  One load instruction reads 4 rows x 256 contiguous bytes: lane l holds
// bytes 64 (l & 3) + 16 (l >> 4) .. + 15 of row 4 i + (l >> 2 & 3), so the
// product's 16 rows are 4 weight rows x 4 segments of 64 bytes, and the 16 columns
// of B are 4 tokens x the same 4 segments.  Of the sums only those of equal
// segments are wanted: element e = l & 3 of lane l, row 4 i + (l >> 4), token
// 4 v + (l >> 2 & 3); a quad's four lanes hold the four segments of one output.
// The matrix cores do 4 times the useful products, a tenth of their time here;
// in exchange the stream needs no LDS and every load reads whole lines.
// Memory bounds it: one token x 16384 x 8192 takes 21.5 us (6.2 TB/s), the gated
// unit x 28672 x 8192 70 us (6.8 TB/s).
template <int VG>
struct StreamRecord {
    int4v a[4], b[VG];
};

typedef int int4u __attribute__((ext_vector_type(4), aligned(4)));

template <bool GATED, int VG>
__global__ __launch_bounds__(kWave * kI8StreamWaves) void i8_stream_kernel(I8Product p, int type) {
    constexpr int KS = kI8StreamWaves;
    constexpr int kRecordWords = 64;
    constexpr int kOuts = 16 * 4 * VG, OC = GATED ? 8 : 16;
    __shared__ int part[KS][kOuts];
    const int lane = lane_id(), m = lane & 15, g = lane >> 4;
    // the same in every lane: keeps the wave's share of k and its loop scalar
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int64_t n0 = (int64_t)blockIdx.x * OC;
    const int left = (int)min((int64_t)OC, p.rows - n0);
    const int at = (m & 3) * 16 + g * 4;
    const int32_t *wrow[4], *xrow[VG];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int slot = 4 * i + (m >> 2);
        wrow[i] = (GATED && slot >= 8 ? p.w_up : p.w) + (n0 + min(slot % OC, left - 1)) * p.kw;
    }
    bool live[VG];
#pragma unroll
    for (int v = 0; v < VG; ++v) {
        live[v] = 4 * v + (m >> 2) < p.tokens;
        xrow[v] = p.x + (int64_t)min(4 * v + (m >> 2), p.tokens - 1) * p.kw;
    }
    const int all = p.kw / kRecordWords, per_wave = (all + KS - 1) / KS;
    const int first = min(all, wave * per_wave), records = min(all, first + per_wave) - first;
    int4v acc[4][VG];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < VG; ++v) acc[i][v] = int4v{0, 0, 0, 0};
    auto consume = [&](const StreamRecord<VG> &q) {
#pragma unroll
        for (int v = 0; v < VG; ++v) {
            const int4v b = live[v] ? q.b[v] : int4v{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i][v] = __builtin_amdgcn_mfma_i32_16x16x64_i8(q.a[i], b, acc[i][v], 0, 0, 0);
        }
    };
    int c = first * kRecordWords + at;
    pipelined<2, StreamRecord<VG>>(
        records,
        [&]() {
            StreamRecord<VG> q;
#pragma unroll
            for (int i = 0; i < 4; ++i) q.a[i] = __builtin_nontemporal_load((const int4u *)(wrow[i] + c));
#pragma unroll
            for (int v = 0; v < VG; ++v) q.b[v] = *(const int4u *)(xrow[v] + c);
            c += kRecordWords;
            return q;
        },
        consume);
    if (p.kw % kRecordWords && wave == KS - 1) {  // the rest of the row: words past it are zero
        StreamRecord<VG> q;
        auto guarded = [&](const int32_t *row) {
            int4v v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = all * kRecordWords + at + e;
                v[e] = j < p.kw ? row[j < p.kw ? j : 0] : 0;
            }
            return v;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) q.a[i] = guarded(wrow[i]);
#pragma unroll
        for (int v = 0; v < VG; ++v) q.b[v] = guarded(xrow[v]);
        consume(q);
    }
    // each quad adds its output's 4 segments; its first lane publishes the sum
    const int e = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < VG; ++v) {
            const int4v d = acc[i][v];
            int t = e == 0 ? d[0] : e == 1 ? d[1] : e == 2 ? d[2] : d[3];
            t = t + dpp<kDppQuadSwap1>(t);
            t = t + dpp<kDppQuadSwap2>(t);
            if (e == 0) part[wave][(4 * v + (m >> 2)) * 16 + 4 * i + g] = t;
        }
    __syncthreads();
    for (int o = threadIdx.x; o < OC * 4 * VG; o += kWave * KS) {
        const int t = o / OC, r = o % OC;
        if (t >= p.tokens || r >= left) continue;
        int sum = 0, up = 0;
#pragma unroll
        for (int q = 0; q < KS; ++q) {
            sum += part[q][t * 16 + r];
            if (GATED) up += part[q][t * 16 + 8 + r];
        }
        const int64_t n = n0 + r;
        const float xs = p.x_scale ? p.x_scale[t] : 1.0f;
        float y = (float)sum * p.w_scale[n] * xs;
        if (GATED) y = act_value(p.act, y) * ((float)up * p.up_scale[n] * xs);
        else if (p.bias) y = y + p.bias[n];
        store1(p.out, type, t * p.out_stride + n, y);
    }
}

template <typename C>
__global__ __launch_bounds__(C::NW * kWave, 1) void i8_tile_kernel(I8Product p, int type) {
    __shared__ __align__(1024) char lds[C::kLds];
    uint32_t ch, tok;
    tile_of(blockIdx.x, count_of(p.rows, C::OUT_CH), count_of(p.tokens, C::TK), 8, ch, tok);
    TileLoop<C> loop(p, lds, (int64_t)ch * C::OUT_CH, (int64_t)tok * C::TK);
    int4v acc[C::WT][C::XT];
#pragma unroll
    for (int i = 0; i < C::WT; ++i)
#pragma unroll
        for (int x = 0; x < C::XT; ++x) acc[i][x] = int4v{};
    const int steps = p.kw / 32;
    loop.run(acc, 0, steps, p.tokens <= C::TK && steps > 0 ? (int)(ch * 5 % steps) : 0, p.kw % 32 != 0);
    const bool whole = p.out_stride % 4 == 0 && (uintptr_t)p.out % (4 * element_bytes(type)) == 0;
    const int64_t n = TileOut<C>::out_channel(loop), left = p.rows - n;
    float ws[4], us[4], bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t m = min(n + e, (int64_t)p.rows - 1);
        ws[e] = p.w_scale[m];
        us[e] = C::GATED ? p.up_scale[m] : 1.0f;
        bias[e] = !C::GATED && p.bias ? p.bias[m] : 0.0f;
    }
    typedef TileOut<C> Out;
    const int64_t start = Out::first_token(loop) * p.out_stride + n, by = Out::PER * p.out_stride;
    Out::each(loop, acc, [&](const typename Out::Pass (&pass)[Out::GROUP]) {
        float y[Out::GROUP][4];
        bool live[Out::GROUP];
#pragma unroll
        for (int j = 0; j < Out::GROUP; ++j) {
            live[j] = pass[j].live;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[j][e] = (float)pass[j].one[e] * ws[e] * pass[j].scale;
        }
        if constexpr (C::GATED) {
            with_activation(p.act, [&](auto act) {
#pragma unroll
                for (int j = 0; j < Out::GROUP; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[j][e] = act_value(decltype(act)::value, y[j][e]) *
                                  ((float)pass[j].two[e] * us[e] * pass[j].scale);
            });
        } else if (p.bias) {
#pragma unroll
            for (int j = 0; j < Out::GROUP; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[j][e] = y[j][e] + bias[e];
        }
        store4_each(p.out, type, start + pass[0].i * by, by, left, whole, live, y);
    });
}

// Few tiles: the waves of a workgroup split k, each running its own tile loop over
// its own rings with no barrier, and add their sums at the end.  A CU then has four
// chains of loads in flight instead of one: 32 tokens x 500 channels x k 16000
// took 22 us with the tile shared by the waves, 11 us so.
template <typename C>
__global__ __launch_bounds__(C::kShape.waves() * kWave, 1) void i8_split_kernel(I8Product p, int type) {
    constexpr int S = C::kShape.split, ROW = C::CH * 4;  // bytes of a token's sums
    static_assert(C::CH == 32 && C::kLds >= C::TK * ROW, "the sums fit the rings");
    __shared__ __align__(1024) char lds[S * C::kLds];
    uint32_t ch, tok;
    tile_of(blockIdx.x, count_of(p.rows, C::OUT_CH), count_of(p.tokens, C::TK), 8, ch, tok);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave)), lane = lane_id();
    TileLoop<C> loop(p, lds + wave * C::kLds, (int64_t)ch * C::OUT_CH, (int64_t)tok * C::TK);
    int4v acc[C::WT][C::XT];
#pragma unroll
    for (int i = 0; i < C::WT; ++i)
#pragma unroll
        for (int x = 0; x < C::XT; ++x) acc[i][x] = int4v{0, 0, 0, 0};
    const int all = p.kw / 32, begin = (int)((int64_t)all * wave / S), end = (int)((int64_t)all * (wave + 1) / S);
    loop.run(acc, begin, end - begin, end > begin ? (int)(ch * 5 % (end - begin)) : 0, wave == S - 1 && p.kw % 32 != 0);
    // the sums of token t, chunks of four channels, at chunk c ^ (t & 7) of its row
#pragma unroll
    for (int i = 0; i < C::WT; ++i)
#pragma unroll
        for (int x = 0; x < C::XT; ++x) {
            const int t = x * 16 + (lane & 15);
            *(int4v *)(loop.lds + t * ROW + (((i * 4 + (lane >> 4)) ^ (t & 7)) << 4)) = acc[i][x];
        }
    __syncthreads();
    constexpr int LANES = C::OUT_CH / 4;
    const bool whole = p.out_stride % 4 == 0 && (uintptr_t)p.out % (4 * element_bytes(type)) == 0;
    for (int o = threadIdx.x; o < C::TK * LANES; o += S * kWave) {
        const int t = o / LANES, c = o % LANES;
        const int64_t n = loop.n0 + 4 * c, left = p.rows - n, token = loop.t0 + t;
        if (left <= 0 || token >= p.tokens) continue;
        int4v one = {0, 0, 0, 0}, two = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < S; ++w) {
            one += *(const int4v *)(lds + w * C::kLds + t * ROW + ((c ^ (t & 7)) << 4));
            if constexpr (C::GATED) two += *(const int4v *)(lds + w * C::kLds + t * ROW + (((c + LANES) ^ (t & 7)) << 4));
        }
        const float xs = p.x_scale ? p.x_scale[token] : 1.0f;
        float y[4], u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t m = n + min((int64_t)e, left - 1);
            y[e] = (float)one[e] * p.w_scale[m] * xs;
            u[e] = C::GATED ? (float)two[e] * p.up_scale[m] * xs : 0.0f;
            if (!C::GATED && p.bias) y[e] = y[e] + p.bias[m];
        }
        if constexpr (C::GATED)
            with_activation(p.act, [&](auto act) {
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = act_value(decltype(act)::value, y[e]) * u[e];
            });
        store4(p.out, type, token * p.out_stride + n, left, whole, y);
    }
}

template <bool GATED, int SHAPE = 0>
void launch_tile(int shape, dim3 grid, dim3 block, const I8Product &p, int type, hipStream_t stream) {
    if constexpr (SHAPE < kI8TileCount + kI8SplitCount) {
        if (shape != SHAPE) return launch_tile<GATED, SHAPE + 1>(shape, grid, block, p, type, stream);
        typedef TileConfig<GATED, SHAPE> C;
        if constexpr (SHAPE < kI8TileCount) hipLaunchKernelGGL((i8_tile_kernel<C>), grid, block, 0, stream, p, type);
        else hipLaunchKernelGGL((i8_split_kernel<C>), grid, block, 0, stream, p, type);
    }
}

template <bool GATED>
hipError_t run(const loom_launch_config &cfg, const I8Product &p, int type, hipStream_t stream) {
    const dim3 grid(cfg.workgroups[0]), block(cfg.workgroup_size[0]);
    if (p.tokens > i8_stream_max_tokens(GATED)) {
        launch_tile<GATED>(i8_tile_choice(p.rows, 4 * (int64_t)p.kw, p.tokens, GATED, true), grid, block, p, type, stream);
        return hipGetLastError();
    }
    switch (i8_stream_groups(p.tokens)) {
        case 1: hipLaunchKernelGGL((i8_stream_kernel<GATED, 1>), grid, block, 0, stream, p, type); break;
        case 2: hipLaunchKernelGGL((i8_stream_kernel<GATED, 2>), grid, block, 0, stream, p, type); break;
        default:
            if constexpr (!GATED) hipLaunchKernelGGL((i8_stream_kernel<false, 4>), grid, block, 0, stream, p, type);
    }
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
