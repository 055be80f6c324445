// i8_gated_backward.hpp -- gradients of the gated projection.
//
// With g, u the two scaled products (recomputed: the int32 sums are exact, so
// they are the forward pass's bits) and d the gradient of the output,
//     dg = d * u * act'(g),   du = d * act(g)
//     d_x[t][i]         = sum_f dg[t][f] gate_scale[f] w_gate[f][i] + du[t][f] up_scale[f] w_up[f][i]
//     d_gate_scale[f]   = sum_t dg[t][f] acc_gate[t][f] x_scale[t]
//     d_up_scale[f]     = sum_t du[t][f] acc_up[t][f] x_scale[t]
// d_x is the gradient with respect to the dequantised activation x * x_scale.
//
// The coefficients dg gate_scale and du up_scale go to memory as 16-bit limbs, and
// d_x is a product of them on the matrix cores: the int8 weights are exact in
// bfloat16 and in float16, so only the coefficients are rounded.  For float16
// gradients they are two bfloat16 limbs (16 bits or more), for float32 ones three
// (exact).  For bfloat16 gradients, which have 8 bits themselves, they are one
// float16 limb: 11 bits, an eighth of what the last rounding of d_x loses, at the
// cost of one limb.  Its exponents have the range of one power of two for each
// token: float16 is full down to 2^-20 of the token's largest coefficient, and
// what is below is off by at most 2^-30 of that coefficient.  All sums are f32.
// (One bfloat16 limb made the whole 2 to 4 % faster, and its rounding was as large as
// d_x's own: 0.0023 of d_x against 0.0017.  Two would double d_x's products.)
#pragma once

#include <algorithm>

#include "i8_tiles.hpp"

namespace loom {

namespace {

// A coefficient's limbs: the leading 8 bits by truncation, so that neither the
// first nor the difference can overflow, and so on; the last is rounded.  What is
// not finite has no second limb.
__device__ __forceinline__ uint32_t bf16_bits(float c) { return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)c); }
template <int LIMBS>
__device__ __forceinline__ void limbs_of(float c, uint32_t (&limb)[LIMBS]) {
#pragma unroll
    for (int i = 0; i + 1 < LIMBS; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, c) & 0xFFFF0000u;
        limb[i] = b >> 16;
        c = (b & 0x7F800000u) == 0x7F800000u ? 0.0f : c - __builtin_bit_cast(float, b);
    }
    limb[LIMBS - 1] = bf16_bits(c);
}

// The power of two that a block of float16 coefficients is divided by: 2^(8 e) with
// the block's largest magnitude, `top`, in 2^6 .. 2^14 of it, so that blocks that
// are as large as each other mostly have the same.  Infinite ones get the largest.
__device__ __forceinline__ int block_exponent(float top) {
    const int e = ((int)(__builtin_bit_cast(uint32_t, top) >> 23) - 133) >> 3;
    return e < -15 ? -15 : e;
}
__device__ __forceinline__ float power_of_two(int e) { return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23); }
__device__ __forceinline__ uint32_t f16_bits(float c) { return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)c); }

struct Coefficients {
    const void *d_out;
    int64_t d_stride;
    int type;
    uint16_t *coef;  // [limbs][tokens][2][padded], or NULL
    int64_t padded;
    int8_t *exponents;  // [tokens][blocks of a wave's channels], one limb only
    int64_t blocks;
    float *sums;     // [token tiles][2][rows]
    float *scale[2]; // one token tile: the scale gradients themselves, or NULL
    bool whole_sums; // there is one token tile
};

// The largest of non-negative numbers over each aligned group of 4, 8 or 16 lanes.
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
    v = fmaxf(v, dpp<kDppQuadSwap1>(v));
    v = fmaxf(v, dpp<kDppQuadSwap2>(v));
    if constexpr (LANES >= 8) v = fmaxf(v, dpp<kDppHalfMirror>(v));
    if constexpr (LANES >= 16) v = fmaxf(v, dpp<kDppMirror>(v));
    static_assert(LANES == 4 || LANES == 8 || LANES == 16, "the steps above");
    return v;
}

// Both products again, then d_x's coefficients and the tile's terms of the scale
// gradients: a lane adds the terms of its four channels over its tokens, then the
// lanes of the same channels, then the waves, always in the same order.
template <typename C, int LIMBS>
__global__ __launch_bounds__(C::NW * kWave, 1) void coefficients_kernel(I8Product p, Coefficients o) {
    typedef TileOut<C, true> Out;
    __shared__ __align__(1024) char lds[C::kLds];
    uint32_t ch, tok;
    tile_of(blockIdx.x, count_of(p.rows, C::OUT_CH), count_of(p.tokens, C::TK), 8, ch, tok);
    TileLoop<C> loop(p, lds, (int64_t)ch * C::OUT_CH, (int64_t)tok * C::TK);
    int4v acc[C::WT][C::XT];
#pragma unroll
    for (int i = 0; i < C::WT; ++i)
#pragma unroll
        for (int x = 0; x < C::XT; ++x) acc[i][x] = int4v{0, 0, 0, 0};
    const int steps = p.kw / 32;
    loop.run(acc, 0, steps, p.tokens <= C::TK && steps > 0 ? (int)(ch * 5 % steps) : 0, p.kw % 32 != 0);
    const bool whole = o.d_stride % 4 == 0 && (uintptr_t)o.d_out % (4 * element_bytes(o.type)) == 0;
    const int64_t n = Out::out_channel(loop), left = p.rows - n;
    float ws[4], us[4], tg[4] = {}, tu[4] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t m = min(n + e, (int64_t)p.rows - 1);
        ws[e] = p.w_scale[m];
        us[e] = p.up_scale[m];
    }
    // four neighbours of d_out as they are in memory (past the last token, its)
    const bool direct = whole && left >= 4;
    const int64_t t1 = Out::first_token(loop);
    auto fetch = [&](int pass, int4v (&into)[Out::PASSES]) {
        const int64_t t = t1 + pass * Out::PER, last = p.tokens - 1;
        if (o.type == LOOM_F32 && direct) {
#pragma unroll
            for (int i = 0; i < Out::PASSES; ++i)
                into[i] = *(const int4v *)((const float *)o.d_out + min(t + i * Out::PER, last) * o.d_stride + n);
        } else if (direct) {
#pragma unroll
            for (int i = 0; i < Out::PASSES; ++i) {
                const uint2v v =
                    *(const uint2v *)((const uint16_t *)o.d_out + min(t + i * Out::PER, last) * o.d_stride + n);
                into[i] = int4v{(int)v.x, (int)v.y, 0, 0};
            }
        } else {
#pragma unroll
            for (int i = 0; i < Out::PASSES; ++i) {
                float d[4];
                load4(o.d_out, o.type, min(t + i * Out::PER, last) * o.d_stride + n, left, false, d);
#pragma unroll
                for (int e = 0; e < 4; ++e) into[i][e] = __builtin_bit_cast(int, d[e]);
            }
        }
    };
    const int64_t start = t1 * 2 * o.padded + n, by = Out::PER * 2 * o.padded, limb = (int64_t)p.tokens * 2 * o.padded;
    Out::each(loop, acc, fetch, [&](const typename Out::Pass (&pass)[Out::GROUP]) {
        if (n >= o.padded) return;
        float cg[Out::GROUP][4], cu[Out::GROUP][4];
        with_activation(p.act, [&](auto act) {
#pragma unroll
            for (int j = 0; j < Out::GROUP; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w = (uint32_t)pass[j].more[e / 2] >> (16 * (e % 2));
                    const float d = o.type == LOOM_F32 || !direct ? __builtin_bit_cast(float, (int)pass[j].more[e])
                                    : o.type == LOOM_F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)w)
                                                         : __builtin_bit_cast(float, w << 16);
                    const float a = (float)pass[j].one[e], b = (float)pass[j].two[e], xs = pass[j].scale;
                    const float g = a * ws[e] * xs, u = b * us[e] * xs;
                    float value, slope;
                    act_value_slope(decltype(act)::value, g, value, slope);
                    const bool in = pass[j].live && e < left;
                    const float dg = in ? d * u * slope : 0.0f, du = in ? d * value : 0.0f;
                    tg[e] = tg[e] + (in ? dg * (a * xs) : 0.0f);
                    tu[e] = tu[e] + (in ? du * (b * xs) : 0.0f);
                    cg[j][e] = dg * ws[e];
                    cu[j][e] = du * us[e];
                }
        });
        if (!o.coef) return;
#pragma unroll
        for (int j = 0; j < Out::GROUP; ++j) {
            uint32_t lg[4][LIMBS], lu[4][LIMBS];
            int exponent = 0;
            if constexpr (LIMBS == 1) {
                // a block: the wave's channels of the token, in Out::LANES neighbouring lanes
                float top = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < left) top = fmaxf(top, fmaxf(fabsf(cg[j][e]), fabsf(cu[j][e])));
                exponent = block_exponent(lanes_max<Out::LANES>(top));
            }
            const float scale = power_of_two(-8 * exponent);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float g = e < left ? cg[j][e] : 0.0f, u = e < left ? cu[j][e] : 0.0f;
                if constexpr (LIMBS == 1) {
                    lg[e][0] = f16_bits(g * scale);
                    lu[e][0] = f16_bits(u * scale);
                } else {
                    limbs_of<LIMBS>(g, lg[e]);
                    limbs_of<LIMBS>(u, lu[e]);
                }
            }
            if (!pass[j].live) continue;
            if (LIMBS == 1 && loop.lane % Out::LANES == 0 && n < p.rows)
                o.exponents[(t1 + (pass[0].i + j) * Out::PER) * o.blocks + n / Out::OC] = (int8_t)exponent;
#pragma unroll
            for (int i = 0; i < LIMBS; ++i) {
                uint16_t *row = o.coef + start + (pass[0].i + j) * by + i * limb;
                *(uint2v *)row = uint2v{lg[0][i] | lg[1][i] << 16, lg[2][i] | lg[3][i] << 16};
                *(uint2v *)(row + o.padded) = uint2v{lu[0][i] | lu[1][i] << 16, lu[2][i] | lu[3][i] << 16};
            }
        }
    });
    // the last tile of a row clears what is left of its padding
    const int64_t end = loop.n0 + C::OUT_CH, pad = o.padded - end;
    if (o.coef && end >= p.rows && pad > 0) {
        const int64_t words = pad / 2, tokens = min((int64_t)C::TK, p.tokens - loop.t0);
        for (int64_t i = threadIdx.x; i < 2 * LIMBS * tokens * words; i += C::NW * kWave) {
            const int64_t row = i / words, part = row / tokens, t = loop.t0 + row % tokens;  // part: 2 limb + up
            uint16_t *at = o.coef + (((part / 2) * p.tokens + t) * 2 + part % 2) * o.padded + end;
            ((uint32_t *)at)[i % words] = 0;
        }
    }
    if (!o.sums && !o.scale[0] && !o.scale[1]) return;
    __syncthreads();
    // [waves][2][OC] sums
    float *mine = (float *)lds + loop.wave * 2 * Out::OC;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int far = Out::LANES; far < kWave; far *= 2) {
            tg[e] = tg[e] + __shfl_xor(tg[e], far);
            tu[e] = tu[e] + __shfl_xor(tu[e], far);
        }
        if (loop.lane < Out::LANES) {
            mine[4 * loop.lane + e] = tg[e];
            mine[Out::OC + 4 * loop.lane + e] = tu[e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * C::OUT_CH; i += C::NW * kWave) {
        const int which = i / C::OUT_CH, c = i % C::OUT_CH, wm = c / Out::OC;
        if (loop.n0 + c >= p.rows) continue;
        float sum = 0.0f;
#pragma unroll
        for (int wn = 0; wn < C::WN; ++wn)
            sum = sum + ((const float *)lds)[((wn * C::WM + wm) * 2 + which) * Out::OC + c % Out::OC];
        if (!o.whole_sums) o.sums[((int64_t)tok * 2 + which) * p.rows + loop.n0 + c] = sum;
        else if (o.scale[which]) o.scale[which][loop.n0 + c] = sum;
    }
}

__global__ __launch_bounds__(256) void scale_gradients_kernel(const float *__restrict__ sums, int64_t tiles,
                                                              int64_t rows, float *__restrict__ d_gate,
                                                              float *__restrict__ d_up) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= 2 * rows) return;
    float sum = 0.0f;
    for (int64_t i = 0; i < tiles; ++i) sum = sum + sums[i * 2 * rows + c];
    float *to = c < rows ? d_gate : d_up;
    if (to) to[c < rows ? c : c - rows] = sum;
}

// One power of two a token for its float16 coefficients: the largest of its blocks'.
// Blocks that were divided by another are divided again, in place (a few in ten where
// the coefficients are alike, as their powers are 2^8 apart); a workgroup a token.
// 1003 tokens x 11008 channels: 7 us; 2048 x 28672: 41 us (one place of four channels
// at a time 10 and 54 us).
__global__ __launch_bounds__(256) void token_powers_kernel(uint16_t *coef, int64_t padded, int64_t tokens, int rows,
                                                           const int8_t *__restrict__ exponents, int block,
                                                           float *__restrict__ powers) {
    __shared__ int tops[4];
    const int blocks = (rows + block - 1) / block, shift = __builtin_ctz(block);  // block: a power of two
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        const int8_t *mine = exponents + t * blocks;
        int top = -15;
        for (int b = threadIdx.x; b < blocks; b += 256) top = max(top, (int)mine[b]);
#pragma unroll
        for (int far = 1; far < kWave; far *= 2) top = max(top, __shfl_xor(top, far));
        if (lane_id() == 0) tops[threadIdx.x / kWave] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, tops[i]);
        __syncthreads();
        if (threadIdx.x == 0) powers[t] = power_of_two(8 * top);
        // PLACES places of four channels at once, their reads in flight together
        constexpr int PLACES = 8;
        typedef _Float16 Half4 __attribute__((ext_vector_type(4)));
        for (int first = 4 * threadIdx.x; first < rows; first += 4 * 256 * PLACES) {
            int by[PLACES];
            Half4 c[PLACES][2];
#pragma unroll
            for (int i = 0; i < PLACES; ++i) {
                const int n = first + i * 4 * 256;
                by[i] = n < rows ? top - mine[n >> shift] : 0;
            }
            Half4 *at = (Half4 *)(coef + 2 * t * padded + first), *up = (Half4 *)((uint16_t *)at + padded);
#pragma unroll
            for (int i = 0; i < PLACES; ++i)
                if (by[i]) {
                    c[i][0] = at[i * 256];
                    c[i][1] = up[i * 256];
                }
#pragma unroll
            for (int i = 0; i < PLACES; ++i)
                if (by[i]) {
                    const float scale = power_of_two(by[i] > 15 ? -120 : -8 * by[i]);
                    auto divided = [&](Half4 h) {
                        return Half4{(_Float16)((float)h[0] * scale), (_Float16)((float)h[1] * scale),
                                     (_Float16)((float)h[2] * scale), (_Float16)((float)h[3] * scale)};
                    };
                    at[i * 256] = divided(c[i][0]);
                    up[i * 256] = divided(c[i][1]);
                }
        }
    }
}

// ---------------------------------------------------------------- d_x
// D[i][t] = sum_f w[f][i] c[t][f] over the gate rows f, then the up rows, in steps
// of 64 rows.  LDS holds a ring of steps: 64 rows x TI bytes of weights and, for
// each limb, TK tokens x 64 coefficients, 16-byte chunk c of row r at
// slot c ^ (r % chunks) in both.  The A operand (16 columns i, 8 neighbouring f a
// lane) is the weights' transpose: ds_read_b64_tr_b8 hands each lane of a group of
// 16 one column of 8 rows x 16 bytes.  Those 8 bytes become bfloat16, or float16 for
// one limb, while the products of the fragment before run: 8 conversions and 4 byte
// permutes, or 2 exclusive ors, 4 byte permutes and 4 subtractions, for XT * LIMBS
// products.
// 2048 tokens x 28672 channels x k 8192 in tiles of 256 x 256, one limb: 1.38 to 1.52
// ms (1.3 to 1.4 PFLOP/s), the matrix cores 66 % busy at the clock their power leaves.
// With bfloat16's conversions, at 1.40 to 1.45 ms: waves of 128 x 128, which convert
// every weight fragment twice, took 1.55 ms; without the conversions it would have
// taken 1.3 ms, without its loads 1.2.
template <int SHAPE, int LIMBS_>
struct DxConfig {
    static constexpr I8DxShape kShape = kI8Dx[SHAPE];
    static constexpr int LIMBS = LIMBS_, WM = kShape.wm, WN = kShape.wn, WT = kShape.it, XT = kShape.xt;
    static constexpr bool GATED = false;
    static constexpr int NW = WM * WN, TI = kShape.columns(), TK = kShape.tokens();
    static constexpr int kRing = kShape.ring(LIMBS), kBytes = kShape.step_bytes(LIMBS), kLds = kRing * kBytes;
    static constexpr int kChunks = TI / 16;                         // of a weight row
    static constexpr int WJ = 64 * TI / 1024 / NW, XJ = LIMBS * TK / 8 / NW, J = WJ + XJ;
    static_assert(64 * TI % (1024 * NW) == 0 && TK % (8 * NW) == 0 && kRing * J <= 63, "whole, countable loads");
    static_assert(kLds <= 160 * 1024, "LDS");
};

struct DxOperands {
    const int8_t *w[2];   // gate, up
    const uint16_t *coef;
    int64_t padded;
    int64_t rows, k;
    int splits;
    void *out;            // d_x, or the f32 parts [splits][tokens][k]
    int type;
};

// FRESH: a was converted just before (two wait states from a vector instruction).
template <bool HALF, bool FRESH>
__device__ __forceinline__ void mfma_16(int4v &acc, int4v a, int4v b) {
    if constexpr (HALF && FRESH) asm("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    else if constexpr (HALF) asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    else if constexpr (FRESH) asm("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    else asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}

template <typename C>
struct DxFragments {
    uint2v a[C::WT];
    int4v b[C::LIMBS][C::XT];
};

template <typename C>
struct DxLoop {
    const I8Product &p;
    const DxOperands &o;
    char *lds;
    int64_t n0, t0;  // first column, first token
    int lane, wave, wm, wn;

    __device__ DxLoop(const I8Product &p_, const DxOperands &o_, char *lds_, int64_t n0_, int64_t t0_)
        : p(p_), o(o_), lds(lds_), n0(n0_), t0(t0_), lane(lane_id()),
          wave(__builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave))) {
        wm = wave % C::WM;
        wn = wave / C::WM;
    }

    // Fragment Q of the half step kk (channels 32 kk ..), in the order of need:
    // a[0], b[..][0 .. XT), a[1 .. WT).
    static constexpr int kB = C::LIMBS * C::XT, kReads = C::WT + kB;
    template <int Q>
    __device__ __forceinline__ void read(DxFragments<C> &f, int at, int kk) const {
        if constexpr (Q > 0 && Q <= kB) {
            constexpr int l = (Q - 1) / C::XT, x = (Q - 1) % C::XT;
            const int off = (lane & 15) * 128 + ((((lane >> 4) ^ (lane & 7)) << 4) ^ (kk * 64));
            f.b[l][x] = *(const int4v *)(lds + at + 64 * C::TI + l * C::TK * 128 + (wn * C::XT + x) * 2048 + off);
        } else {
            constexpr int i = Q ? Q - kB : 0;
            // lane j of a group of 16 reads half j & 1 of row j >> 1 of its 8
            const int row = kk * 32 + (lane >> 4) * 8 + (lane >> 1 & 7);
            const int slot = (wm * C::WT + i) ^ (row % C::kChunks);
            const char *from = lds + at + row * C::TI + slot * 16 + (lane & 1) * 8;
            typedef int int2v __attribute__((ext_vector_type(2)));
            f.a[i] = __builtin_bit_cast(uint2v, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                                                    (__attribute__((address_space(3))) int2v *)(from)));
        }
    }

    // Elements 2 J, 2 J + 1 of a fragment as bfloat16: an int8's f32 has no bits
    // below the upper half.  As float16: 0x6400 + b is 1024 + b, and b the element
    // plus 128.
    template <int J>
    __device__ static __forceinline__ uint32_t pair(uint2v raw) {
        const uint32_t w = raw[J / 2];
        if constexpr (C::LIMBS == 1) {
            typedef _Float16 Half2 __attribute__((ext_vector_type(2)));
            const uint32_t b = __builtin_amdgcn_perm(0x64646464u, w ^ 0x80808080u, J % 2 ? 0x04030402u : 0x04010400u);
            return __builtin_bit_cast(uint32_t, __builtin_bit_cast(Half2, b) - Half2{(_Float16)1152, (_Float16)1152});
        }
        const float lo = (float)(int8_t)(w >> (16 * (J % 2))), hi = (float)(int8_t)(w >> (16 * (J % 2) + 8));
        return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
    }

    __device__ __forceinline__ void run(int4v (&acc)[C::WT][C::XT], int first, int count) {
        const int64_t half = o.padded / kI8ChannelPad;  // steps of a matrix
        const int left_t = (int)min((int64_t)C::TK, p.tokens - t0);
        // this lane's place in each of its wave's direct loads; columns past the
        // row read its neighbour's and tokens past the end the last one's, whose
        // sums are not stored
        int wo[C::WJ], xo[C::XJ];
        constexpr int ROWS = 1024 / C::TI;  // weight rows of one load
#pragma unroll
        for (int j = 0; j < C::WJ; ++j) {
            const int row = (wave + C::NW * j) * ROWS + lane / C::kChunks;
            wo[j] = row * (int)o.k + ((lane % C::kChunks) ^ (row % C::kChunks)) * 16;
        }
#pragma unroll
        for (int j = 0; j < C::XJ; ++j) {
            const int row = ((wave + C::NW * j) * 8) % C::TK + (lane >> 3);
            xo[j] = min(row, left_t - 1) * (int)(4 * o.padded) + ((lane & 7) ^ (lane >> 3)) * 16;
        }
        const int at = lds_address(lds) + wave * 1024;
        const uint16_t *tokens = o.coef + t0 * 2 * o.padded;
        const int last = first + count;
        // Load j of step s.  Weight rows past the matrix are past the buffer and
        // read as 0 (their coefficients are 0 too); a step past the end reads
        // nothing.
        auto load = [&](int s, int place, int j) {
            const bool up = s >= half;
            const int64_t f0 = (up ? s - half : s) * kI8ChannelPad;
            const int to = at + place + C::NW * j * 1024;
            if (j < C::WJ) {
                const int64_t from = f0 * o.k + n0;
                int4v r = buffer_over((up ? o.w[1] : o.w[0]) + from, s < last ? o.rows * o.k - from : 0);
                load_to_lds(r, wo[j < C::WJ ? j : 0], 0, to);
            } else {
                const int limb = (C::NW * (j - C::WJ) * 8) / C::TK;
                int4v r = buffer_over(tokens + (int64_t)limb * p.tokens * 2 * o.padded,
                                      s < last ? 4 * o.padded * left_t : 0);
                load_to_lds(r, xo[j < C::WJ ? 0 : j - C::WJ], s * 128, to);
            }
        };
        constexpr int J = C::J, Q = C::WT * C::XT * C::LIMBS, GROUP = C::XT * C::LIMBS, R = Q / 2, L = Q * 5 / 8;
        constexpr int W = Q >= 64 ? Q - L + Q * 7 / 8 : Q - L;
        constexpr auto place_of = [](int j) { return L + j * W / J; };
        constexpr int EARLY = [](auto place) { int n = 0; while (n < J && place(n) < Q) ++n; return n; }(place_of);
#pragma unroll
        for (int s = 0; s < C::kRing; ++s)
            each_index<J>([&](auto j) { load(first + s, s * C::kBytes, decltype(j)::value); });
        wait_loads<(C::kRing - 1) * J>();
        barrier();
        DxFragments<C> f0, f1;
        each_index<kReads>([&](auto r) { read<decltype(r)::value>(f0, 0, 0); });
        uint32_t ready[2][4];  // the fragment in use, and the next, widened
        each_index<4>([&](auto j) { ready[0][decltype(j)::value] = pair<decltype(j)::value>(f0.a[0]); });
        // Half a step: the products of f, while the next half's fragments are read
        // into g and converted.
        auto product = [&](auto at_q, const DxFragments<C> &f, const DxFragments<C> &g) {
            constexpr int q = decltype(at_q)::value, i = q / GROUP, in = q % GROUP;
            // the pairs of the next fragment, spread over this one's products
            each_index<4>([&](auto at_j) {
                constexpr int j = decltype(at_j)::value;
                if constexpr (j * (GROUP < 8 ? GROUP : 8) / 4 / (GROUP < 8 ? 1 : 2) == in)
                    ready[(i + 1) % 2][j] = pair<j>(i + 1 < C::WT ? f.a[i + 1 < C::WT ? i + 1 : 0] : g.a[0]);
            });
            const int4v a = {(int)ready[i % 2][0], (int)ready[i % 2][1], (int)ready[i % 2][2], (int)ready[i % 2][3]};
            mfma_16<C::LIMBS == 1, in == 0>(acc[i][in % C::XT], a, f.b[in / C::XT][in % C::XT]);
        };
        static_assert(C::WT % 2 == 0, "a half step ends on the pair it began on");
        int s = first, here = 0;
        do {
            each_index<Q>([&](auto at_q) {
                constexpr int q = decltype(at_q)::value;
                each_index<kReads>([&](auto at_r) {
                    constexpr int r = decltype(at_r)::value;
                    if constexpr (r * R / kReads == q) read<r>(f1, here, 1);
                });
                if constexpr (q == L) {
                    wait_lds();
                    barrier();
                }
                each_index<J>([&](auto at_j) {
                    constexpr int j = decltype(at_j)::value;
                    if constexpr (place_of(j) == q) load(s + C::kRing, here, j);
                });
                product(at_q, f0, f1);
                pin();
            });
            const int left = here;
            here = here == C::kLds - C::kBytes ? 0 : here + C::kBytes;
            wait_loads<(C::kRing - 2) * J + EARLY>();
            barrier();
            each_index<Q>([&](auto at_q) {
                constexpr int q = decltype(at_q)::value;
                each_index<kReads>([&](auto at_r) {
                    constexpr int r = decltype(at_r)::value;
                    if constexpr (r * (Q * 3 / 4) / kReads == q) read<r>(f0, here, 0);
                });
                each_index<J>([&](auto at_j) {
                    constexpr int j = decltype(at_j)::value;
                    if constexpr (place_of(j) == Q + q) load(s + C::kRing, left, j);
                });
                product(at_q, f1, f0);
                pin();
            });
        } while (++s < last);
        wait_loads<0>();
        wait_lds();
        settle(acc);
    }
};

template <typename C>
__global__ __launch_bounds__(C::NW * kWave, 1) void d_x_kernel(I8Product p, DxOperands o) {
    __shared__ __align__(1024) char lds[C::kLds];
    uint32_t ch, tok;
    tile_of(blockIdx.x, count_of((int)o.k, C::TI), count_of(p.tokens, C::TK), 8, ch, tok);
    DxLoop<C> loop(p, o, lds, (int64_t)ch * C::TI, (int64_t)tok * C::TK);
    int4v acc[C::WT][C::XT];
#pragma unroll
    for (int i = 0; i < C::WT; ++i)
#pragma unroll
        for (int x = 0; x < C::XT; ++x) acc[i][x] = int4v{0, 0, 0, 0};
    const int steps = (int)(2 * o.padded / kI8ChannelPad);
    const int first = (int)((int64_t)steps * blockIdx.y / o.splits), last = (int)((int64_t)steps * (blockIdx.y + 1) / o.splits);
    loop.run(acc, first, last - first);
    const bool parts = o.splits > 1;
    const int type = parts ? (int)LOOM_F32 : o.type;
    void *out = parts ? (void *)((float *)o.out + (int64_t)blockIdx.y * p.tokens * o.k) : o.out;
    const bool whole = o.k % 4 == 0 && (uintptr_t)out % (4 * element_bytes(type)) == 0;
    const int64_t n = TileOut<C>::out_channel(loop), left = o.k - n;
    typedef TileOut<C> Out;
    const int64_t start = Out::first_token(loop) * o.k + n, by = Out::PER * o.k;
    Out::each(loop, acc, [&](const typename Out::Pass (&pass)[Out::GROUP]) {
        float y[Out::GROUP][4];
        bool live[Out::GROUP];
#pragma unroll
        for (int j = 0; j < Out::GROUP; ++j) {
            live[j] = pass[j].live;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[j][e] = __builtin_bit_cast(float, (int)pass[j].one[e]);
                if (C::LIMBS == 1) y[j][e] = y[j][e] * pass[j].scale;  // the token's power of two
            }
        }
        store4_each(out, type, start + pass[0].i * by, by, left, whole, live, y);
    });
}

__global__ __launch_bounds__(256) void add_parts_kernel(const float *__restrict__ parts, int splits, int64_t count,
                                                        void *d_x, int type, bool whole) {
    // count is a multiple of 4
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < count; i += (int64_t)gridDim.x * 1024) {
        float4v sum = *(const float4v *)(parts + i);
        int s = 1;
        for (; s + 8 <= splits; s += 8) {  // eight loads in flight, added in order
            float4v part[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) part[j] = *(const float4v *)(parts + (s + j) * count + i);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = sum + part[j];
        }
        for (; s < splits; ++s) sum = sum + *(const float4v *)(parts + s * count + i);
        const float y[4] = {sum[0], sum[1], sum[2], sum[3]};
        store4(d_x, type, i, 4, whole, y);
    }
}

__global__ __launch_bounds__(256) void zero_kernel(void *d_x, int type, int64_t count, bool whole) {
    const float y[4] = {};
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < count; i += (int64_t)gridDim.x * 1024)
        store4(d_x, type, i, 4, whole, y);
}

template <int LIMBS, int SHAPE = 0>
void launch_coefficients(int shape, dim3 grid, dim3 block, const I8Product &p, const Coefficients &o,
                         hipStream_t stream) {
    if constexpr (SHAPE < kI8TileCount) {
        if (shape != SHAPE) return launch_coefficients<LIMBS, SHAPE + 1>(shape, grid, block, p, o, stream);
        hipLaunchKernelGGL((coefficients_kernel<TileConfig<true, SHAPE>, LIMBS>), grid, block, 0, stream, p, o);
    }
}

template <int SHAPE, int LIMBS>
void launch_d_x(const I8DxPlan &plan, const I8Product &p, const DxOperands &o, hipStream_t stream) {
    typedef DxConfig<SHAPE, LIMBS> C;
    hipLaunchKernelGGL((d_x_kernel<C>), dim3((uint32_t)plan.tiles, plan.splits), dim3(C::NW * kWave), 0, stream, p, o);
}

template <int LIMBS>
hipError_t run_backward(const loom_launch_config &cfg, const I8Product &p, const void *d_out, int type, int64_t d_stride,
               void *d_x, float *d_gate, float *d_up, void *workspace, hipStream_t stream) {
    const int64_t rows = p.rows, tokens = p.tokens, k = 4 * (int64_t)p.kw;
    const I8BackwardSpace space = i8_backward_space(rows, k, tokens, type);
    const int shape = i8_tile_choice(rows, k, tokens, true, false);
    const int64_t padded = ceil_of(rows, kI8ChannelPad) * kI8ChannelPad;
    const bool scales = (d_gate || d_up) && rows > 0, inputs = d_x && tokens > 0 && k > 0;
    uint16_t *coef = inputs ? (uint16_t *)workspace : nullptr;
    float *sums = scales ? (float *)((char *)workspace + space.sums) : nullptr;
    const bool one = tokens > 0 && tokens <= kI8Tiles[shape].tokens();
    const int block = kI8Tiles[shape].wave_channels();
    const int64_t blocks = ceil_of(rows, block);
    int8_t *exponents = (int8_t *)workspace + space.exponents;
    float *powers = (float *)((char *)workspace + space.powers);
    if (tokens > 0 && rows > 0) {
        const Coefficients o = {d_out, d_stride, type, coef, padded, exponents, blocks, one ? nullptr : sums,
                                {one ? d_gate : nullptr, one ? d_up : nullptr}, one};
        launch_coefficients<LIMBS>(shape, dim3(cfg.workgroups[0]), dim3(cfg.workgroup_size[0]), p, o, stream);
    }
    if (scales && !one)
        hipLaunchKernelGGL(scale_gradients_kernel, dim3((uint32_t)((2 * rows + 255) / 256)), dim3(256), 0, stream,
                           sums, ceil_of(tokens, kI8Tiles[shape].tokens()), rows, d_gate, d_up);
    if (!inputs) return hipGetLastError();
    const int64_t count = tokens * k;
    const bool whole = (uintptr_t)d_x % (4 * element_bytes(type)) == 0;
    const dim3 flat((uint32_t)std::min<int64_t>((count / 4 + 255) / 256, 1 << 16));
    if (rows == 0) {
        hipLaunchKernelGGL(zero_kernel, flat, dim3(256), 0, stream, d_x, type, count, whole);
        return hipGetLastError();
    }
    const I8DxPlan plan = i8_dx_plan(rows, k, tokens, type);
    float *parts = (float *)((char *)workspace + space.parts);
    if (LIMBS == 1)
        hipLaunchKernelGGL(token_powers_kernel, dim3((uint32_t)std::min<int64_t>(tokens, 1 << 20)), dim3(256), 0, stream,
                           coef, padded, tokens, p.rows, exponents, block, powers);
    I8Product plain = p;
    plain.x_scale = LIMBS == 1 ? powers : nullptr;  // the tile's output applies it
    const DxOperands o = {{(const int8_t *)p.w, (const int8_t *)p.w_up}, coef, padded, rows, k, plan.splits,
                          plan.splits > 1 ? (void *)parts : d_x, type};
    switch (plan.shape) {
        case 0:
            if constexpr (LIMBS == 1) launch_d_x<0, LIMBS>(plan, plain, o, stream);
            break;
        case 1: launch_d_x<1, LIMBS>(plan, plain, o, stream); break;
        case 2: launch_d_x<2, LIMBS>(plan, plain, o, stream); break;
        default: launch_d_x<3, LIMBS>(plan, plain, o, stream);
    }
    if (plan.splits > 1)
        hipLaunchKernelGGL(add_parts_kernel, flat, dim3(256), 0, stream, parts, plan.splits, count, d_x, type, whole);
    return hipGetLastError();
}

}  // namespace

}  // namespace loom
