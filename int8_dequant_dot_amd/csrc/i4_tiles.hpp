// i4_tiles.hpp -- the tile of the 4-bit products: activations, packed weights and
// scales through LDS, group sums on the int8 matrix cores.
#pragma once

#include "i4_common.hpp"
#include "i8_tiles.hpp"

namespace loom {

// global_load_dwordx4 ... lds: lane l's 16 bytes at its address land at LDS byte
// at + 16 l.  Not counted by the compiler, as load_to_lds.
__device__ __forceinline__ void gather_to_lds(const void *from, int at) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, off"
        :
        : "s"(at), "v"(from)
        : "memory", "m0");
}

// A tile is 32 XT WN tokens x 32 WM WT channels (gated: half of them gate, half up rows
// of the same channels), computed by WN x WM waves, each XT x WT blocks of 32 x 32.
// A operand: 32 tokens, B: 32 channels; lane l holds 16 elements of token or channel
// l & 31, half h = l >> 5 of the product's 32, and of the sums channel l & 31, tokens
// 8 (r >> 2) + 4 h + (r & 3).
//
// A step is PARTS (1 or 2) parts of 128 elements of k, SUBS groups of 128 / SUBS each
// (with one, part of a longer group).  Product i of a part's four takes the 16-element pieces
// piece(i, 0) and piece(i, 1): both halves of 32 neighbours where SUBS is 4, else a
// half each of two 32s, whose weights are then one read for both.
//
// LDS holds two steps: rows of 128 PARTS bytes of activations and of 64 PARTS bytes of
// weights, filled by direct loads; 16-byte piece c of row r sits at slot c ^ swizzle(r),
// so that fragment reads meet no bank twice.
//
// The vector unit is the fuller one, 69 % of the cycles at 4096 tokens x 8192 channels x k
// 28672, the matrix cores 41 %: each sum of 32 x 32 x 128 takes a conversion and a multiply-add
// (256 of the 530 vector instructions of a wave's step of 256), its weights three instructions
// for two registers; the rest is waits, of two waves a SIMD that meet at every step.  That size
// takes 1.05 to 1.10 ms in groups of 128 (1750 to 1830 TOP/s; without loads 0.88 to 0.93), 1.95
// in groups of 32, four times the conversions.  Not kept there: weights straight from memory to registers
// (1.64 ms: a line for every 16 bytes of a lane), reads that wait for the barrier of their
// own step (1.24 ms), scales read by each lane (1.21 ms), one wave a SIMD with twice the
// tokens (1.22 ms: the sums go through the accumulation registers), 128 x 128 tiles, two a
// CU (1.17 ms).
template <int SHAPE, int SUBS_, bool GATED_>
struct I4Tile {
    static constexpr I4TileShape kShape = i4_tile_shape(SHAPE, GATED_);
    static constexpr int XT = kShape.xt, WN = kShape.wn, WM = kShape.wm, WT = kShape.wt, SUBS = SUBS_, PARTS = kShape.parts;
    static constexpr bool GATED = GATED_;
    static constexpr int NW = WM * WN, TK = kShape.tokens(), CH = kShape.channels(), OUT_CH = GATED ? CH / 2 : CH;
    static constexpr int kRowX = 128 * PARTS, kRowW = 64 * PARTS, kBytesX = TK * kRowX, kBytesW = CH * kRowW, kStep = kBytesX + kBytesW;
    static constexpr int kBytesS = PARTS * SUBS * CH * 4;  // a step's scales, as f32
    static constexpr int kLds = 2 * (kStep + kBytesS);
    static constexpr int XJ = kBytesX / 1024 / NW, WJ = kBytesW / 1024 / NW;  // direct loads a wave and step
    static constexpr int SJ = PARTS * CH < NW * kWave ? 1 : PARTS * CH / (NW * kWave);  // channels' parts whose scales a thread loads
    static constexpr int PER = 4 / SUBS;                      // products of a group within a part
    static_assert(kBytesX % (1024 * NW) == 0 && kBytesW % (1024 * NW) == 0 && (SJ == 1 || PARTS * CH % (NW * kWave) == 0) &&
                      (!GATED || WT == 2), "whole loads a wave");
    static_assert(kLds * kShape.split == kShape.lds(SUBS) && kShape.lds(SUBS) <= 160 * 1024, "the launch's LDS");
    static __device__ constexpr int swizzle_x(int r) { return r & (8 * PARTS - 1); }
    static __device__ constexpr int swizzle_w(int r) { return PARTS == 2 ? r & 7 : (r >> 1) & 3; }
    static __device__ constexpr int piece(int i, int h) { return SUBS == 4 ? 2 * i + h : 4 * (i >> 1) + 2 * h + (i & 1); }
};

template <typename C, int ST>
struct I4TileLoop {
    const I4Product &p;
    char *lds;
    int lane, wave, wm, wn, half, m;  // wave: of the tile
    int64_t t0, n0;    // first token (routed row), first output channel of the workgroup
    int rows, expert;  // rows of the tile

    float acc[C::XT][C::WT][16];

    // LDS weight row r -> its matrix (gated: 32 gate rows and the same 32 up rows a
    // wave) and its row there.
    __device__ __forceinline__ bool is_up(int r) const { return C::GATED && (r & 32); }
    __device__ __forceinline__ int64_t weight_row(int r) const {
        const int64_t n = n0 + (C::GATED ? (r >> 6) * 32 + (r & 31) : r);
        return (int64_t)expert * p.rows + min(n, (int64_t)p.rows - 1);
    }
    __device__ __forceinline__ const int32_t *matrix(bool up) const { return up ? p.w_up : p.w; }
    __device__ __forceinline__ const void *scales(bool up) const { return up ? p.up_scale : p.w_scale; }

    // Waves of one tile meet; a wave with a tile of its own goes on.
    __device__ __forceinline__ static void meet() {
        if constexpr (C::NW > 1) barrier();
    }

    // Adds the products of the steps begin .. begin + steps - 1, and where `tail` those
    // past the last whole step.  row_of(r): the row of x for row r of the tile.
    template <typename RowOf>
    __device__ __forceinline__ void run(int begin, int steps, bool tail, RowOf &&row_of) {
#pragma unroll
        for (int x = 0; x < C::XT; ++x)
#pragma unroll
            for (int w = 0; w < C::WT; ++w)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[x][w][r] = 0.0f;
        const int64_t kb = (int64_t)p.chunks * 32;
        const char *from_x[C::XJ], *from_w[C::WJ];
#pragma unroll
        for (int j = 0; j < C::XJ; ++j) {
            const int slot = (wave + C::NW * j) * kWave + lane, r = slot / (8 * C::PARTS), c = slot % (8 * C::PARTS);
            from_x[j] = (const char *)p.x + row_of(min(r, rows - 1)) * kb + ((c ^ C::swizzle_x(r)) << 4);
        }
#pragma unroll
        for (int j = 0; j < C::WJ; ++j) {
            const int slot = (wave + C::NW * j) * kWave + lane, r = slot / (4 * C::PARTS), c = slot % (4 * C::PARTS);
            from_w[j] = (const char *)matrix(is_up(r)) + weight_row(r) * (kb / 2) + ((c ^ C::swizzle_w(r)) << 4);
        }
        const int at = lds_address(lds) + wave * 1024;
        // load J of step s, into that place
        auto load = [&](auto at_j, int64_t s, int place) {
            constexpr int j = decltype(at_j)::value, k = j < C::XJ ? 0 : j - C::XJ;
            const int to = at + (place & 1) * C::kStep;
            if constexpr (j < C::XJ) gather_to_lds(from_x[j] + (begin + s) * C::kRowX, to + C::NW * j * 1024);
            else gather_to_lds(from_w[k] + (begin + s) * C::kRowW, to + C::kBytesX + C::NW * k * 1024);
        };
        // Scales: read by every wave that uses them, a line for each lane and two bytes, they
        // took 110 of 1200 us at 4096 x 8192 x 28672.  Each thread reads those of one channel
        // and part of a step, and they wait in LDS.
        typedef typename ElementOf<ST>::type Scale;
        typedef Scale Scales __attribute__((ext_vector_type(C::SUBS), aligned(sizeof(Scale))));
        float *const held = (float *)(lds + 2 * C::kStep);
        const Scale *my_scales[C::SJ];
        Scales coming[C::SJ];
        const int tid = wave * kWave + lane;
#pragma unroll
        for (int j = 0; j < C::SJ; ++j) {
            const int r = (tid + j * C::NW * kWave) / C::PARTS % C::CH;
            my_scales[j] = (const Scale *)scales(is_up(r)) + weight_row(r) * p.groups;
        }
        auto fetch_scales = [&](int s) {
            s = begin + min(s, steps - 1);
            const int h = s * C::PARTS + tid % C::PARTS, g = C::SUBS > 1 ? h * C::SUBS : (4 * h) >> p.chunk_shift;
#pragma unroll
            for (int j = 0; j < C::SJ; ++j) coming[j] = *(const Scales *)(my_scales[j] + g);
        };
        auto keep_scales = [&](int s) {
#pragma unroll
            for (int j = 0; j < C::SJ; ++j) {
                const int r = (tid + j * C::NW * kWave) / C::PARTS % C::CH;
                float *to = held + ((s & 1) * C::PARTS + tid % C::PARTS) * (C::SUBS * C::CH) + r;
#pragma unroll
                for (int u = 0; u < C::SUBS; ++u) to[u * C::CH] = (float)coming[j][u];
            }
        };
        if (steps > 0) {
            float scale[C::WT][C::SUBS];
            fetch_scales(0);
            keep_scales(0);
            each_index<C::XJ + C::WJ>([&](auto j) { load(j, 0, 0); });
            each_index<C::XJ + C::WJ>([&](auto j) { load(j, min(1, steps - 1), 1); });
            wait_loads<C::XJ + C::WJ>();
            wait_lds();
            meet();
            constexpr int WL = C::SUBS == 4 ? 4 : 2;
            int4v a[4], raw[C::WT][WL], b[C::WT][4];
            const char *base_x = lds + (wn * C::XT * 32 + m) * C::kRowX;
            const char *base_w = lds + C::kBytesX + (wm * C::WT * 32 + m) * C::kRowW;
            // fragments of part h of the step at that place
            auto read_a = [&](int place, int h, int x, int i) {
                a[i] = *(const int4v *)(base_x + place + x * 32 * C::kRowX + (((8 * h + C::piece(i, half)) ^ C::swizzle_x(m)) << 4));
            };
            auto read_w = [&](int place, int h) {
#pragma unroll
                for (int w = 0; w < C::WT; ++w)
#pragma unroll
                    for (int i = 0; i < WL; ++i) {
                        const int c = 4 * h + (C::SUBS == 4 ? i : 2 * i + half);
                        raw[w][i] = *(const int4v *)(base_w + place + w * 32 * C::kRowW + ((c ^ C::swizzle_w(m)) << 4));
                    }
            };
            auto unpack = [&](int w, int i) {
                if constexpr (C::SUBS == 4) b[w][i] = half ? i4_high(raw[w][i]) : i4_low(raw[w][i]);
                else b[w][i] = i & 1 ? i4_high(raw[w][i >> 1]) : i4_low(raw[w][i >> 1]);
            };
            read_w(0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                read_a(0, 0, 0, i);
#pragma unroll
                for (int w = 0; w < C::WT; ++w) unpack(w, i);
            }
            pin();
            int16v sum[2];
            for (int s = 0; s < steps; ++s) {
                const int place = (s & 1) * C::kStep, other = C::kStep - place;
                const int64_t after = min(s + 2, steps - 1);  // past the end the last step again
                fetch_scales(s + 1);
                const float *my = held + (s & 1) * (C::PARTS * C::SUBS * C::CH) + wm * C::WT * 32 + m;
                // units of PER products that end a group's part, block by block; while one is
                // multiplied the sums of the one before are converted, scaled and added, and in
                // the last blocks the next part's fragments are read and unpacked into the
                // registers that the products leave
                constexpr int UNITS = C::XT * C::WT * C::SUBS;
                each_index<C::PARTS>([&](auto at_h) {
                    constexpr int h = decltype(at_h)::value, then_h = (h + 1) % C::PARTS;
                    constexpr bool last = h == C::PARTS - 1;
                    const int then = last ? other : place;
#pragma unroll
                    for (int w = 0; w < C::WT; ++w)
#pragma unroll
                        for (int u = 0; u < C::SUBS; ++u) scale[w][u] = my[(h * C::SUBS + u) * C::CH + w * 32];
                    each_index<UNITS + 1>([&](auto at_u) {
                        constexpr int u = decltype(at_u)::value, sub = u % C::SUBS, w = u / C::SUBS % C::WT,
                                      x = u / C::SUBS / C::WT;
                        each_index<C::PER>([&](auto at_i) {
                            constexpr int i = decltype(at_i)::value, q = sub * C::PER + i;
                            if constexpr (x == C::XT - 1 && w == 0 && q == 0) {
                                if constexpr (last) {
                                    // all fragments of this step are in registers, and this wave's part
                                    // of the next step is in LDS: once every wave is here the next step
                                    // may be read and this one's place filled
                                    keep_scales(s + 1);
                                    wait_loads<0>();
                                    wait_lds();
                                    meet();
                                }
                                read_w(then, then_h);
                            }
                            if constexpr (u < UNITS)
                                sum[u & 1] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[q], b[w][q], i == 0 ? int16v{} : sum[u & 1], 0, 0, 0);
                            if constexpr (u < UNITS && w == C::WT - 1) {
                                if constexpr (x + 1 < C::XT) read_a(place, h, x + 1, q);
                                else read_a(then, then_h, 0, q);
                            }
                            if constexpr (u < UNITS && x == C::XT - 1 && w == C::WT - 1) {
#pragma unroll
                                for (int y = 0; y < C::WT; ++y) unpack(y, q);
                            }
                            if constexpr (last && u < UNITS && x == C::XT - 1) {
                                constexpr int n = w * 4 + q, J = C::XJ + C::WJ;
                                each_index<J>([&](auto at_j) {
                                    if constexpr (decltype(at_j)::value * 4 * C::WT / J == n) load(at_j, after, s);
                                });
                            }
                            if constexpr (u > 0) {
                                constexpr int v = u - 1, vs = v % C::SUBS, vw = v / C::SUBS % C::WT, vx = v / C::SUBS / C::WT;
#pragma unroll
                                for (int r = i * 16 / C::PER; r < (i + 1) * 16 / C::PER; ++r)
                                    acc[vx][vw][r] = __builtin_fmaf((float)sum[v & 1][r], scale[vw][vs], acc[vx][vw][r]);
                            }
                            pin();
                        });
                    });
                });
            }
            wait_loads<0>();
        }
        // the rest of k, less than a step, in parts of a group and at most 128
        constexpr int kPart = 4 / C::SUBS;
        for (int c0 = tail ? p.chunks / (4 * C::PARTS) * (4 * C::PARTS) : p.chunks; c0 < p.chunks; c0 += kPart) {
            const int c1 = min(c0 + kPart, p.chunks), g = c0 >> p.chunk_shift;
#pragma unroll
            for (int x = 0; x < C::XT; ++x) {
                const int4v *xr = (const int4v *)((const char *)p.x + row_of(min((wn * C::XT + x) * 32 + m, rows - 1)) * kb);
                int16v sum[C::WT] = {};
                for (int c = c0; c < c1; ++c)
#pragma unroll
                    for (int w = 0; w < C::WT; ++w) {
                        const int64_t row = weight_row((wm * C::WT + w) * 32 + m);
                        const int4v v = ((const int4v *)matrix(C::GATED && w))[row * p.chunks + c];
                        sum[w] = __builtin_amdgcn_mfma_i32_32x32x32_i8(xr[2 * c + half], half ? i4_high(v) : i4_low(v), sum[w], 0, 0, 0);
                    }
#pragma unroll
                for (int w = 0; w < C::WT; ++w) {
                    const float scale = scale_at<ST>(scales(C::GATED && w), weight_row((wm * C::WT + w) * 32 + m) * p.groups + g);
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[x][w][r] = __builtin_fmaf((float)sum[w][r], scale, acc[x][w][r]);
                }
            }
        }
    }

    // Stores the sums r0 .. r0 + N - 1 of each block.  scale_of(r): x_scale of row r of the tile, which
    // may be subnormal: the factor kI4Unit would cost it bits, so the sums take it.
    template <int N, typename ScaleOf>
    __device__ __forceinline__ void store(int type, int r0, ScaleOf &&scale_of) {
        if (type == LOOM_F32) store_as<N>((float *)p.out, r0, scale_of);
        else if (type == LOOM_F16) store_as<N>((_Float16 *)p.out, r0, scale_of);
        else store_as<N>((__bf16 *)p.out, r0, scale_of);
    }
    template <int N, typename T, typename ScaleOf>
    __device__ __forceinline__ void store_as(T *out, int r0, ScaleOf &&scale_of) {
        constexpr int OUT = C::GATED ? 1 : C::WT;  // of a wave's blocks of channels
        const int64_t n = n0 + (C::GATED ? wm * 32 + m : wm * C::WT * 32 + m);
        float bias[OUT];
#pragma unroll
        for (int w = 0; w < OUT; ++w)
            bias[w] = !C::GATED && p.bias ? p.bias[(int64_t)expert * p.rows + min(n + w * 32, (int64_t)p.rows - 1)] : 0.0f;
#pragma unroll
        for (int x = 0; x < C::XT; ++x) {
            const int first = (wn * C::XT + x) * 32;
            if (first >= rows) return;
            const float xs = scale_of(min(first + m, rows - 1));
            T *to = out + (t0 + first + 4 * half) * p.out_stride + n;
            const int limit = rows - first - 4 * half;
            float y[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int r = r0 + e;
                y[e] = __shfl(xs, 8 * (r >> 2) + (r & 3) + 4 * half);
            }
            if constexpr (C::GATED) {
                with_activation(p.act, [&](auto act) {
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        acc[x][0][e] = act_value(decltype(act)::value, acc[x][0][e] * kI4Unit * y[e]) * (acc[x][C::WT - 1][e] * kI4Unit * y[e]);
                });
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int r = r0 + e, row = 8 * (r >> 2) + (r & 3);
                T *at = to + row * p.out_stride;
#pragma unroll
                for (int w = 0; w < OUT; ++w) {
                    float v = acc[x][w][e];
                    if constexpr (!C::GATED) v = v * kI4Unit * y[e];
                    if (!C::GATED && p.bias) v = v + bias[w];
                    if (row < limit && n + w * 32 < p.rows) at[w * 32] = (T)v;
                }
            }
        }
    }
};

}  // namespace loom
