// i8_tiles.hpp -- the int8 matrix-core tile loop of the product, the gated
// projection and its gradients: LDS tiles filled by direct loads, read as
// v_mfma_i32_16x16x64_i8 fragments.
#pragma once

#include "ffn_common.hpp"

namespace loom {

// ---------------------------------------------------------------- direct loads into LDS
// buffer_load_dwordx4 ... lds: lane l's 16 bytes at base + voff + soff land at
// LDS byte at + 16 l, with no register in between.  The compiler does not
// count these loads, so every wait for them is written out (wait_loads); they
// retire in order.
__device__ __forceinline__ void load_to_lds(int4v rsrc, int voff, int soff, int at) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds"
        :
        : "s"(at), "v"(voff), "s"(rsrc), "s"(soff)
        : "memory", "m0");
}
template <int LEFT>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(LEFT) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }
__device__ __forceinline__ void barrier() {
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
}
// Instructions keep their order across it.
__device__ __forceinline__ void pin() { __builtin_amdgcn_sched_barrier(0); }

// A raw buffer over `bytes` bytes from base (capped: offsets are 32 bits).
__device__ __forceinline__ int4v buffer_over(const void *base, int64_t bytes) {
    const uint64_t b = (uint64_t)(uintptr_t)base;
    const uint32_t size = bytes > 0xFFFFFFFFll ? 0xFFFFFFFFu : (uint32_t)bytes;
    int4v r;
    r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    r.y = __builtin_amdgcn_readfirstlane((int)((uint32_t)(b >> 32) & 0xFFFFu));
    r.z = __builtin_amdgcn_readfirstlane((int)size);
    r.w = 0x00020000;
    return r;
}

__device__ __forceinline__ int lds_address(const void *p) {
    return __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p);
}

// body(0), body(1), .. body(N - 1) with each index a compile-time constant.
template <int N> struct Index { static constexpr int value = N; };
template <int N, int I = 0, typename Body>
__device__ __forceinline__ void each_index(Body &&body) {
    if constexpr (I < N) {
        body(Index<I>{});
        each_index<N, I + 1>(body);
    }
}

// acc += a * b in the accumulation registers.  Written out, because the
// compiler, given accumulators that fill that half of the register file, moves
// them through the other half in every step; it does not know the result's
// latency, so the sums may be read only behind settle().
__device__ __forceinline__ void mfma(int4v &acc, int4v a, int4v b) {
    asm("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
// keep(): the sums from token block FROM on stay in those registers up to here.
template <int FROM = 0, int N, int M>
__device__ __forceinline__ void keep(int4v (&acc)[N][M]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int x = FROM; x < M; ++x) asm volatile("" : "+a"(acc[i][x]));
}
template <int N, int M>
__device__ __forceinline__ void settle(int4v (&acc)[N][M]) {
    pin();
    asm volatile("s_nop 15\n\ts_nop 15" : "+a"(acc[0][0]));
    keep(acc);
    pin();
}

// ---------------------------------------------------------------- the order of the tiles
// Workgroup b runs on XCD b % 8, each with its own L2, so every XCD takes one
// contiguous run of a tile order in which `high` token tiles alternate fastest:
// its 32 CUs then work on a compact rectangle of the output and share its
// weight and activation rows.
__device__ __forceinline__ uint32_t count_of(int n, int tile) { return ((uint32_t)n + tile - 1) / tile; }
__device__ __forceinline__ void tile_of(uint32_t block, uint32_t ch_tiles, uint32_t tok_tiles, uint32_t high,
                                        uint32_t &ch, uint32_t &tok) {
    const uint32_t total = ch_tiles * tok_tiles, q = total / 8, r = total % 8;
    const uint32_t xcd = block % 8, local = block / 8;
    const uint32_t i = xcd * q + min(xcd, r) + local;
    const uint32_t panel = i / (high * ch_tiles), in = i - panel * high * ch_tiles;
    const uint32_t h = min(high, tok_tiles - panel * high);
    tok = panel * high + in % h;
    ch = in / h;
}

// ---------------------------------------------------------------- the tile
// A workgroup computes CH = WM * WT * 16 channels (gated: half of them gate,
// half up rows of the same channels) x TK = WN * XT * 16 tokens with WM x WN
// waves, each WT x XT blocks of 16 x 16.  A operand: 16 weight rows, B: 16
// tokens; lane l holds 16 bytes of row (l & 15) at byte 16 (l >> 4) of a
// 64-byte half step, and of the sums channels 4 (l >> 4) + e of token l & 15.
//
// A step is 128 bytes of k.  LDS holds a ring of kRingW steps of CH rows x 128 bytes
// of weights and one of kRingX steps of TK rows of activations;
// 16-byte chunk c of row r sits at slot c ^ (r & 7) of that row, so the direct
// loads (8 rows x 128 contiguous bytes each) read whole lines and the 16-row
// fragment reads meet no bank twice.
//
// The 256 x 256 shape has four waves of 128 x 128 rather than eight of 128 x 64:
// half the LDS reads a product.  At 4096 tokens x 8192 channels x k 28672 it takes
// 690 us (2780 TOP/s), with the matrix cores 72 % busy at the 1.6 to 2.0 GHz that
// the card's power leaves; without its loads it would take 560 us, without any
// memory access 515 us.  Not kept: the loads of a step issued in a burst (750 us:
// the waves wait for the address path and stop multiplying), a ring of five
// 64-byte steps (764 us: twice the cache lines touched a byte), 32 x 32 x 32
// products in it (803 us: twice the accumulator traffic a product), a ring of
// three steps of weights (700 us).
template <bool GATED_, int SHAPE>
struct TileConfig {
    static constexpr I8TileShape kShape = kI8Tiles[SHAPE];
    static constexpr bool GATED = GATED_;
    static constexpr int WM = kShape.wm, WN = kShape.wn, WT = kShape.wt, XT = kShape.xt;
    static constexpr int kRingW = kShape.ring_w, kRingX = kShape.ring_x;
    static constexpr int NW = WM * WN, CH = WM * WT * 16, TK = WN * XT * 16;
    static constexpr int OUT_CH = GATED ? CH / 2 : CH;  // channels of the output
    static constexpr int kBytesW = CH * 128, kBytesX = TK * 128;  // one step
    static constexpr int kStartX = kRingW * kBytesW, kLds = kStartX + kRingX * kBytesX;  // of one tile
    static constexpr int WJ = CH / 8 / NW, XJ = TK / 8 / NW;  // direct loads a wave and step
    static_assert(CH % (8 * NW) == 0 && TK % (8 * NW) == 0 && (!GATED || WT % 2 == 0), "whole loads a wave");
    static_assert(kLds * kShape.split == kShape.lds() && kShape.lds() <= 160 * 1024, "the launch's LDS");
    static_assert(kRingX >= 2 && kRingW >= kRingX && kRingW * WJ + kRingX * XJ <= 63, "the loads in flight can be counted");
};

template <typename C>
struct TileFragments {
    int4v a[C::WT], b[C::XT];
};

template <typename C>
struct TileLoop {
    const I8Product &p;
    char *lds;
    int64_t n0, t0;  // first output channel, first token
    int lane, wave, wm, wn;

    __device__ TileLoop(const I8Product &p_, char *lds_, int64_t n0_, int64_t t0_)
        : p(p_), lds(lds_), n0(n0_), t0(t0_), lane(lane_id()),
          wave(C::NW > 1 ? __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave)) : 0) {
        wm = wave % C::WM;
        wn = wave / C::WM;
    }
    // Waves of one tile meet; a wave with a tile of its own goes on.
    __device__ __forceinline__ static void meet() {
        if constexpr (C::NW > 1) barrier();
    }

    // LDS weight row r -> row of its matrix, relative to n0 (gated: the first
    // half of each wave's rows are gate rows, the second the same up rows).
    __device__ static int weight_row(int r) {
        if constexpr (!C::GATED) return r;
        return (r / (C::WT * 16)) * (C::WT * 8) + r % (C::WT * 8);
    }
    __device__ static constexpr bool is_up(int r) { return C::GATED && (r % (C::WT * 16)) >= C::WT * 8; }

    // Fragment Q of half step kk of the step at those places, in the order in which the
    // products need them: a[0], b[0 .. XT), a[1 .. WT).
    static constexpr int kReads = C::WT + C::XT;
    template <int Q>
    __device__ __forceinline__ void read(TileFragments<C> &f, int at_w, int at_x, int kk) const {
        const int off = (lane & 15) * 128 + ((((lane >> 4) ^ (lane & 7)) << 4) ^ (kk * 64));
        if constexpr (Q > 0 && Q <= C::XT) {
            f.b[Q - 1] = *(const int4v *)(lds + at_x + (wn * C::XT + Q - 1) * 2048 + off);
        } else {
            constexpr int i = Q ? Q - C::XT : 0;
            f.a[i] = *(const int4v *)(lds + at_w + (wm * C::WT + i) * 2048 + off);
        }
    }

    // Adds the products of `steps` whole steps from step `begin`, in the order
    // first, first + 1, .. round the end, and where `tail` those of the partly
    // filled step behind the last whole one.
    __device__ __forceinline__ void run(int4v (&acc)[C::WT][C::XT], int begin, int steps, int first, bool tail) {
        const int64_t kb = 4 * (int64_t)p.kw;
        const int4v rw = buffer_over(p.w + n0 * p.kw, (p.rows - n0) * kb);
        const int4v ru = C::GATED ? buffer_over(p.w_up + n0 * p.kw, (p.rows - n0) * kb) : rw;
        const int4v rx = buffer_over(p.x + t0 * p.kw, (p.tokens - t0) * kb);
        const int left_n = (int)min((int64_t)C::OUT_CH, p.rows - n0), left_t = (int)min((int64_t)C::TK, p.tokens - t0);
        // this lane's place in each of its wave's direct loads; rows past the
        // matrices read the last row, and their products are not stored
        int wo[C::WJ], xo[C::XJ];
        const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
        for (int j = 0; j < C::WJ; ++j)
            wo[j] = min(weight_row((wave + C::NW * j) * 8 + (lane >> 3)), left_n - 1) * (int)kb + chunk;
#pragma unroll
        for (int j = 0; j < C::XJ; ++j)
            xo[j] = min((wave + C::NW * j) * 8 + (lane >> 3), left_t - 1) * (int)kb + chunk;
        const int at = lds_address(lds) + wave * 1024;
        int4v rj[C::WJ];
#pragma unroll
        for (int j = 0; j < C::WJ; ++j) rj[j] = C::GATED && is_up((wave + C::NW * j) * 8) ? ru : rw;
        // Load j of the activations of step s, or of its weights, into that place.
        // A step past the end reads nothing: its buffers have size 0, so the loop
        // needs no branch for it.
        auto at_step = [&](int s) { return begin + (s + first >= steps ? s + first - steps : s + first); };
        auto load_x = [&](int s, int place, int j) {
            int4v r = rx;
            r.z = s < steps ? r.z : 0;
            load_to_lds(r, xo[j], at_step(s) * 128, at + place + C::NW * j * 1024);
        };
        auto load_w = [&](int s, int place, int j) {
            int4v r = rj[j];
            r.z = s < steps ? r.z : 0;
            load_to_lds(r, wo[j], at_step(s) * 128, at + place + C::NW * j * 1024);
        };
        constexpr int J = C::WJ + C::XJ, Q = C::WT * C::XT, R = Q / 2, L = Q * 5 / 8;
        // The loads of a step are spread over the rest of the first half and the
        // second: issued in a burst they fill the address path's queue, and the
        // wave that issues them stops multiplying (256 x 256: 750 against 697 us;
        // 128 x 256: 37.2 against 34.9 us at 187 x 11008 x 4096, gated).  Smaller
        // tiles wait for memory instead and issue them at once.  EARLY of them are
        // in the first half.
        constexpr int W = Q >= 32 ? Q - L + Q * 7 / 8 : Q - L;
        constexpr auto place_of = [](int j) { return L + j * W / J; };
        constexpr int EARLY = [](auto place) { int n = 0; while (n < J && place(n) < Q) ++n; return n; }(place_of);
        // Two rounds through one copy of the loop (two copies cost the
        // accumulators their registers): first the rest of k, a partly filled
        // step staged word by word, then the whole steps.
        int round = tail ? 0 : 1;
        if (steps == 0 && round == 1) return;
        do {
            const int count = round == 0 ? 1 : steps;
            if (round == 0) {
                for (int c = C::NW > 1 ? (int)threadIdx.x : lane; c < (C::CH + C::TK) * 8; c += C::NW * kWave) {
                    const int r = c >> 3, q = c & 7;
                    const int32_t *row;
                    if (r < C::CH) row = (is_up(r) ? p.w_up : p.w) + (n0 + min(weight_row(r), left_n - 1)) * p.kw;
                    else row = p.x + (t0 + min(r - C::CH, left_t - 1)) * p.kw;
                    int4v v = {0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at_word = p.kw / 32 * 32 + q * 4 + e;
                        if (at_word < p.kw) v[e] = row[at_word];
                    }
                    *(int4v *)(lds + (r < C::CH ? r * 128 : C::kStartX + (r - C::CH) * 128) + ((q ^ (r & 7)) << 4)) = v;
                }
                wait_lds();
            } else {
                meet();  // every wave has read what the first round left
                // in the order in which the steps before the first would load them
#pragma unroll 1
                for (int s = 0; s < C::kRingW; ++s) {
                    const int sx = s + C::kRingX - C::kRingW;
                    if (sx >= 0)
#pragma unroll
                        for (int j = 0; j < C::XJ; ++j) load_x(sx, C::kStartX + sx * C::kBytesX, j);
#pragma unroll
                    for (int j = 0; j < C::WJ; ++j) load_w(s, s * C::kBytesW, j);
                }
                // what came after x(0), and w(0) where that was later
                wait_loads<(C::kRingX - 1) * J + (C::kRingW > C::kRingX ? C::WJ : 0)>();
            }
            meet();
            TileFragments<C> f0, f1;
            each_index<kReads>([&](auto r) { read<decltype(r)::value>(f0, 0, C::kStartX, 0); });
            const int skip = round == 0 ? steps : 0;  // the first round loads nothing
            int s = 0, here_w = 0, here_x = C::kStartX;
            do {
                // first half: multiply bytes 0-63 and read 64-127 in its first
                // 5/8; then every wave is done with this place and it takes a
                // later step
                each_index<Q>([&](auto at_q) {
                    constexpr int q = decltype(at_q)::value;
                    each_index<kReads>([&](auto at_r) {
                        constexpr int r = decltype(at_r)::value;
                        if constexpr (r * R / kReads == q) read<r>(f1, here_w, here_x, 1);
                    });
                    if constexpr (q == L) {
                        wait_lds();
                        meet();
                    }
                    each_index<J>([&](auto at_j) {
                        constexpr int j = decltype(at_j)::value;
                        if constexpr (place_of(j) == q) {
                            if constexpr (j < C::XJ) load_x(s + C::kRingX + skip, here_x, j);
                            else load_w(s + C::kRingW + skip, here_w, j - C::XJ);
                        }
                    });
                    mfma(acc[q / C::XT][q % C::XT], f0.a[q / C::XT], f0.b[q % C::XT]);
                    pin();
                });
                // second half: multiply bytes 64-127, read the next step's 0-63
                // (after the last step whatever the place holds, unused)
                const int left_w = here_w, left_x = here_x;
                here_w = here_w == (C::kRingW - 1) * C::kBytesW ? 0 : here_w + C::kBytesW;
                here_x = here_x == C::kLds - C::kBytesX ? C::kStartX : here_x + C::kBytesX;
                // what came after x(s + 1), and w(s + 1) where that was later
                wait_loads<(C::kRingX - 2) * J + EARLY + (C::kRingW > C::kRingX ? C::WJ : 0)>();
                meet();
                each_index<Q>([&](auto at_q) {
                    constexpr int q = decltype(at_q)::value;
                    each_index<kReads>([&](auto at_r) {
                        constexpr int r = decltype(at_r)::value;
                        if constexpr (r * (Q * 3 / 4) / kReads == q) read<r>(f0, here_w, here_x, 0);
                    });
                    each_index<J>([&](auto at_j) {
                        constexpr int j = decltype(at_j)::value;
                        if constexpr (place_of(j) == Q + q) {
                            if constexpr (j < C::XJ) load_x(s + C::kRingX + skip, left_x, j);
                            else load_w(s + C::kRingW + skip, left_w, j - C::XJ);
                        }
                    });
                    mfma(acc[q / C::XT][q % C::XT], f1.a[q / C::XT], f1.b[q % C::XT]);
                    pin();
                });
            } while (++s < count);
            wait_loads<0>();
            wait_lds();
        } while (++round < 2 && steps > 0);
        settle(acc);
    }
};

// Hands the tile's sums to `use`, transposed through LDS so that a lane holds
// four neighbouring channels n .. n + 3 of one token (and their up sums, gated),
// n = out_channel(), the same for every pass of a lane, and the lanes beside it the
// channels beside those.  use gets GROUP passes at once, pass i token
// first_token() + i * PER, so that their reads, arithmetic and stores overlap and
// it branches on types and activations once for all of them; passes that are not
// live are past the last token.  Each wave moves its own part through its own
// piece of the LDS, some token blocks at a time; wide stores are whole lines.
// (One pass at a time took 23 us of a 256 x 256 tile.)
//
// FETCH: a pass also gets 16 bytes that belong to its sums, with fetch(first pass,
// into) loading those of one lane for PASSES passes; they are loaded while the
// blocks before are in use, and wait in LDS.
template <typename C, bool FETCH = false>
struct TileOut {
    static constexpr int OC = C::WT * 16 / (C::GATED ? 2 : 1);  // output channels of a wave
    static constexpr int LANES = OC / 4;                        // lanes of one token
    static constexpr int PER = kWave / LANES;                   // tokens of one pass
    static constexpr int ROW = C::WT * 64;                      // bytes of one token's sums in LDS
    static constexpr int HELD = FETCH ? 16 * OC * 4 : 0;        // fetched bytes of a token block
    static constexpr int ROOM = C::kLds / C::NW;                // bytes of LDS a wave
    static constexpr int FIT = (ROOM - 64 * C::XT) / (16 * ROW + HELD);
    // token blocks at a time
    static constexpr int BLOCKS = FIT >= C::XT ? C::XT : FIT >= 4 && C::XT % 4 == 0 ? 4 : FIT >= 2 && C::XT % 2 == 0 ? 2 : 1;
    static constexpr int PASSES = BLOCKS * 16 / PER;
    static_assert(C::XT % BLOCKS == 0 && LANES <= kWave && kWave % LANES == 0 && FIT > 0 && PASSES > 0, "whole passes");

    template <typename Loop>
    static __device__ int64_t out_channel(const Loop &l) {
        return l.n0 + l.wm * OC + 4 * (l.lane % LANES);
    }

    template <typename Loop>
    static __device__ int64_t first_token(const Loop &l) {
        return l.t0 + l.wn * C::XT * 16 + l.lane / LANES;
    }

    static constexpr int GROUP = PASSES % 4 == 0 ? 4 : PASSES % 2 == 0 ? 2 : 1;
    struct Pass {
        int i;          // the same in every lane
        bool live;
        float scale;    // the token's
        int4v one, two, more;
    };

    template <typename Loop, typename Use>
    static __device__ __forceinline__ void each(const Loop &l, int4v (&acc)[C::WT][C::XT], Use &&use) {
        each(l, acc, [](int, int4v (&)[PASSES]) {}, use);
    }

    template <typename Loop, typename Fetch, typename Use>
    static __device__ __forceinline__ void each(const Loop &l, int4v (&acc)[C::WT][C::XT], Fetch &&fetch, Use &&use) {
        char *mine = l.lds + l.wave * ROOM;
        float *scales = (float *)(mine + ROOM - 64 * C::XT);
        int4v *held = (int4v *)(mine + BLOCKS * 16 * ROW) + l.lane;
        const int m = l.lane & 15, g = l.lane >> 4, c = l.lane % LANES, r0 = l.lane / LANES;
        const int64_t first = l.t0 + l.wn * C::XT * 16;
        const int count = (int)min((int64_t)C::XT * 16, l.p.tokens - first);
        int4v next[PASSES];
        if (FETCH && count > 0) fetch(0, next);
        __syncthreads();  // every wave is done with the tile
        for (int i = l.lane; i < count; i += kWave) scales[i] = l.p.x_scale ? l.p.x_scale[first + i] : 1.0f;
        each_index<C::XT / BLOCKS>([&](auto round) {
            constexpr int b = decltype(round)::value * BLOCKS;
            if (count <= b * 16) return;
            keep<b>(acc);
#pragma unroll
            for (int x = 0; x < BLOCKS; ++x)
#pragma unroll
                for (int i = 0; i < C::WT; ++i)
                    *(int4v *)(mine + (x * 16 + m) * ROW + (((i * 4 + g) ^ (m & 7)) << 4)) = acc[i][b + x];
            if constexpr (FETCH) {
#pragma unroll
                for (int i = 0; i < PASSES; ++i) held[i * kWave] = next[i];
                if (b + BLOCKS < C::XT && count > (b + BLOCKS) * 16) fetch((b + BLOCKS) * 16 / PER, next);
            }
            wait_lds();
#pragma unroll 1
            for (int at = 0; at < PASSES; at += GROUP) {
                Pass pass[GROUP];
#pragma unroll
                for (int j = 0; j < GROUP; ++j) {
                    const int r = r0 + (at + j) * PER;
                    const char *row = mine + r * ROW;
                    pass[j].i = b * 16 / PER + at + j;
                    pass[j].live = b * 16 + r < count;
                    pass[j].scale = scales[b * 16 + r];
                    pass[j].one = *(const int4v *)(row + ((c ^ (r & 7)) << 4));
                    if constexpr (C::GATED) pass[j].two = *(const int4v *)(row + (((c + LANES) ^ (r & 7)) << 4));
                    if constexpr (FETCH) pass[j].more = held[(at + j) * kWave];
                }
                use(pass);
            }
            wait_lds();
        });
    }
};

}  // namespace loom
