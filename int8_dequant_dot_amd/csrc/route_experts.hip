// route_experts.hip -- routing of tokens to experts, and its gradient.
//
//     s = softmax(l) or sigmoid(l),   c = s + bias, or l itself without a bias
//     a group's value: the sum of its group_top largest c (without a bias: of s)
//     ids: the top_k largest c of the top_groups best groups, in falling order
//     w = s[ids], divided by their sum where renormalised, times scale
//
// Ties go to the lower index.  Neighbouring choices may differ by less than a
// step of f32, so wherever a choice is computed (and is not a logit itself) its
// order is that of its 64-bit value: waves whose f32 choices lie apart by more
// than their error are done with those; where a sigmoid's do not, a few candidates are
// put in the order of their 64-bit values, and where that is not enough, or the scores
// are a softmax's, the wave computes every choice again in 64 bits.  Weights are f32.
//
// 65536 tokens x 256 experts in f32, the 8 best of 4 of 8 groups by sigmoid and bias, take
// 49 to 59 us, where their 71 MB would take 15.  A wave of four tokens runs 1.3 thousand
// vector instructions, 55 % of the cycles; it has 168 registers, so that three waves a SIMD
// share the waits for chains of cross-lane steps, and 70 scalars that are kept in lanes.  16
// lanes hold a token where there are many (fewer cross-lane steps a token), 64 where there
// are few.  With every choice in 64 bits the same took 190 us.  By its bounds 1.2 % of its
// waves order candidates and one in 8 thousand does all in 64 bits; with a softmax 0.9 % do
// (57 us), and from top_k 13 on, where 16 lanes have no room for candidates, 2 to 2.5 %
// (72 us, 78 at 16).
// The gradient streams: 65536 x 256 bfloat16 logits through the softmax take 19 us (3.7 TB/s).
#include <type_traits>

#include "ffn_common.hpp"

namespace loom {

namespace {

// body(0) .. body(N - 1), each index a constant from the start: arrays that are
// written under conditions in unrolled loops have ended in scratch memory.
template <int N, int I = 0, typename Body>
__device__ __forceinline__ void each(Body &&body) {
    if constexpr (I < N) {
        body(std::integral_constant<int, I>{});
        each<N, I + 1>(body);
    }
}

// ---------------------------------------------------------------- within the lanes of a token
// Step S of a butterfly over aligned groups of 2^LOG lanes: the value of the
// lane (or of a lane with the same partial result) on the other side.
template <int S>
__device__ __forceinline__ int other(int v) {
    if constexpr (S == 0) return dpp<kDppQuadSwap1>(v);
    else if constexpr (S == 1) return dpp<kDppQuadSwap2>(v);
    else if constexpr (S == 2) return dpp<kDppHalfMirror>(v);
    else if constexpr (S == 3) return dpp<kDppMirror>(v);
    else if constexpr (S == 4) return swz16(v);
    else return __builtin_amdgcn_ds_bpermute((lane_id() ^ 32) << 2, v);
}
template <int S>
__device__ __forceinline__ float other(float v) { return __builtin_bit_cast(float, other<S>(__builtin_bit_cast(int, v))); }
template <int S>
__device__ __forceinline__ double other(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)other<S>((int)(uint32_t)b), hi = (uint32_t)other<S>((int)(uint32_t)(b >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int LOG, int S = 0, typename T, typename Op>
__device__ __forceinline__ T fold(T v, Op &&op) {
    if constexpr (S < LOG) return fold<LOG, S + 1>(op(v, other<S>(v)), op);
    else return v;
}
template <int LOG, typename T>
__device__ __forceinline__ T fold_sum(T v) { return fold<LOG>(v, [](T a, T b) { return a + b; }); }
template <int LOG, typename T>
__device__ __forceinline__ T fold_max(T v) { return fold<LOG>(v, [](T a, T b) { return a > b ? a : b; }); }
template <int LOG>
__device__ __forceinline__ int fold_min(int v) { return fold<LOG>(v, [](int a, int b) { return a < b ? a : b; }); }
template <int LOG>
__device__ __forceinline__ int fold_or(int v) { return fold<LOG>(v, [](int a, int b) { return a | b; }); }

__device__ __forceinline__ float load_logit(const void *l, int type, int64_t at) {
    if (type == LOOM_F32) return ((const float *)l)[at];
    if (type == LOOM_F16) return (float)((const _Float16 *)l)[at];
    return (float)((const __bf16 *)l)[at];
}

constexpr float kInf = __builtin_inff();

// The factors of a token's chosen experts, one in each lane that has one: s
// relative to e^shift, 0 where nothing was chosen.  A sigmoid is
// e^min(l, 0) / (1 + e^-|l|), which keeps ratios of vanishing scores.
template <int LOG>
__device__ __forceinline__ float relative_score(int score, float l, bool live, float &shift) {
    const float a = score == LOOM_SIGMOID ? fminf(l, 0.0f) : l;
    shift = fold_max<LOG>(live ? a : -kInf);
    const float e = live ? expf(a - shift) : 0.0f;
    return score == LOOM_SIGMOID ? e / (1.0f + expf(-fabsf(l))) : e;
}

// ---------------------------------------------------------------- the router
// 2^LOG lanes hold a token, R experts a lane, V neighbours at a time: its r-th is
// expert_at(r).  All that a token needs of others is within its wave.
template <int LOG, int R>
struct Held {
    static constexpr int L = 1 << LOG, V = R % 4 == 0 ? 4 : 1;
    typedef float Values __attribute__((ext_vector_type(V)));
    static __device__ __forceinline__ int expert_at(int r, int sub) { return r / V * (L * V) + r % V + sub * V; }
};

// A row's values, `other` past its end; its rows may be aligned to the element only.
template <int LOG, int R, typename T>
__device__ __forceinline__ void load_row(const T *row, int n, int sub, float past, float (&l)[R]) {
    typedef Held<LOG, R> H;
    typedef T Run __attribute__((ext_vector_type(4), aligned(sizeof(T))));
#pragma unroll
    for (int r = 0; r < R; r += H::V) {
        const int e = H::expert_at(r, sub);
        if (H::V == 4 && e + 4 <= n) {
            const Run v = *(const Run *)(row + e);
#pragma unroll
            for (int i = 0; i < H::V; ++i) l[r + i] = (float)v[i];
        } else {
#pragma unroll
            for (int i = 0; i < H::V; ++i) l[r + i] = e + i < n ? (float)row[e + i] : past;
        }
    }
}
template <int LOG, int R>
__device__ __forceinline__ void load_logits(const void *l, int type, int64_t at, int n, int sub, float past, float (&to)[R]) {
    if (type == LOOM_F32) load_row<LOG, R>((const float *)l + at, n, sub, past, to);
    else if (type == LOOM_F16) load_row<LOG, R>((const _Float16 *)l + at, n, sub, past, to);
    else load_row<LOG, R>((const __bf16 *)l + at, n, sub, past, to);
}

template <int LOG, int R, typename T>
__device__ __forceinline__ void store_row_as(T *row, int n, int sub, const float (&y)[R]) {
    typedef Held<LOG, R> H;
    typedef T Run __attribute__((ext_vector_type(4), aligned(sizeof(T))));
#pragma unroll
    for (int r = 0; r < R; r += H::V) {
        const int e = H::expert_at(r, sub);
        if (H::V == 4 && e + 4 <= n) {
            Run v;
#pragma unroll
            for (int i = 0; i < H::V; ++i) v[i] = (T)y[r + i];
            *(Run *)(row + e) = v;
        } else {
#pragma unroll
            for (int i = 0; i < H::V; ++i)
                if (e + i < n) row[e + i] = (T)y[r + i];
        }
    }
}
template <int LOG, int R>
__device__ __forceinline__ void store_row(void *to, int type, int64_t at, int n, int sub, const float (&y)[R]) {
    if (type == LOOM_F32) store_row_as<LOG, R>((float *)to + at, n, sub, y);
    else if (type == LOOM_F16) store_row_as<LOG, R>((_Float16 *)to + at, n, sub, y);
    else store_row_as<LOG, R>((__bf16 *)to + at, n, sub, y);
}

__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// f32 values as whole numbers of the same order (-0 as 0), whose maxima and minima
// need no care for NaNs and fold into cross-lane moves.
__device__ __forceinline__ int key_of(float v) {
    const int b = __builtin_bit_cast(int, v + 0.0f);
    return b ^ (int)((uint32_t)(b >> 31) >> 1);
}
__device__ __forceinline__ float of_key(int k) { return __builtin_bit_cast(float, k ^ (int)((uint32_t)(k >> 31) >> 1)); }
constexpr int kNone = (int)0x807FFFFF;  // key_of(-infinity)
constexpr int kPast = 0x7FFFFFFF;       // past key_of(infinity)
constexpr float kMost = 0x1.fffffep127f;  // the largest finite value

// The two largest of a lane's and of 2^STEPS lanes' values.
__device__ __forceinline__ void keep_two(int v, int &first, int &second) {
    second = max(min(v, first), second);
    first = max(v, first);
}
template <int STEPS, int S = 0>
__device__ __forceinline__ void merge_two(int &first, int &second) {
    if constexpr (S < STEPS) {
        const int a = other<S>(first), b = other<S>(second);
        second = max(max(second, b), min(first, a));
        first = max(first, a);
        merge_two<STEPS, S + 1>(first, second);
    }
}

// Takes the choices of all but the best groups away: a group's value is its largest
// choice, or the sum of its two largest, and a group stays while fewer than top_groups
// are better.  Returns whether the order of 64-bit values keeps the same ones (true where
// COMPUTED is false: logits are what they are): whether the least that one that stays can be
// lies above the most that another can be (groups without a choice apart: it does not matter
// whether they stay).  A group's value is off by its scores' errors, `gap` at most, by the
// choices' roundings, 2^-24 of each, and the sum's, 2^-24 of it: by less than 2^-23 of the
// choices' magnitudes, and twice that leaves room for the bounds' own roundings.
// room: LDS of this token, experts + 3 groups values.
template <bool COMPUTED, int LOG, int R>
__device__ __forceinline__ bool best_groups(const RouteArgs &a, int sub, float *room, int (&c)[R], float gap) {
    typedef Held<LOG, R> H;
    constexpr int L = H::L, B = (R + 3) / 4;
    const int size = a.experts / a.groups;
    int *const ranks = (int *)room + a.experts;
    float *const sizes = room + a.experts + 2 * a.groups;
    auto rank = [&](int g, int first, int second) {
        const bool both = a.group_top > 1 && second > kNone;
        // a sum below the lowest f32 value is not that of a group without choices
        ranks[g] = both ? max(key_of(of_key(first) + of_key(second)), kNone + 1) : first;
        if (COMPUTED) sizes[g] = fabsf(of_key(first)) + (both ? fabsf(of_key(second)) : 0.0f);
    };
    int worst = kPast, best = kNone;
    auto weigh = [&](bool stays, int g) {
        const int mine = ranks[g];
        if (COMPUTED && mine > kNone) {
            // sums beyond the largest f32 value may be anything beyond it
            const float value = of_key(mine), off = fminf(sizes[g], kMost) * 0x1p-22f + gap;
            const float least = value > -kMost ? fminf(value, kMost) - off : -kInf;
            worst = stays ? min(worst, key_of(least)) : worst;
            best = stays ? best : max(best, key_of(value + off));
        }
    };
    if (H::V == 4 && size >= 4 && size <= 4 * L && (size & (size - 1)) == 0) {
        // groups of 4, 8, .. neighbouring experts lie on 1, 2, .. neighbouring lanes
        const int shift = __builtin_ctz(size);
        int group[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            int first = kNone, second = kNone;
#pragma unroll
            for (int i = 0; i < 4; ++i) keep_two(c[min(4 * b + i, R - 1)], first, second);
            switch (shift) {
                case 2: break;
                case 3: merge_two<1>(first, second); break;
                case 4: merge_two<2>(first, second); break;
                case 5: merge_two<3>(first, second); break;
                case 6: merge_two<4>(first, second); break;
                case 7: merge_two<(LOG >= 5 ? 5 : 0)>(first, second); break;
                default: merge_two<(LOG >= 6 ? 6 : 0)>(first, second);
            }
            const int e = H::expert_at(4 * b, sub);
            group[b] = e >> shift;
            if (e < a.experts && (e & (size - 1)) == 0) rank(group[b], first, second);
        }
        wave_fence();
        // a lane a group: how many are better (equal and before it, or greater)
        for (int g = sub; g < a.groups; g += L) {
            const int that = ranks[g];
            int better = 0;
            for (int o = 0; o < a.groups; ++o) better += ranks[o] - (o >= g) >= that;
            weigh(better < a.top_groups, g);
            ranks[a.groups + g] = better;
        }
        wave_fence();
        each<B>([&](auto b) {
            const bool stays = ranks[a.groups + min(group[b], a.groups - 1)] < a.top_groups;
            each<4>([&](auto i) {
                constexpr int r = 4 * decltype(b)::value + decltype(i)::value;
                if constexpr (r < R) {
                    const int own = c[r];
                    c[r] = stays ? own : kNone;
                }
            });
        });
    } else {
        int *const values = (int *)room;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (H::expert_at(r, sub) < a.experts) values[H::expert_at(r, sub)] = c[r];
        wave_fence();
        for (int g = sub; g < a.groups; g += L) {
            int first = kNone, second = kNone;
            for (int i = 0; i < size; ++i) keep_two(values[g * size + i], first, second);
            rank(g, first, second);
        }
        wave_fence();
        // each group's verdict, then each expert's
        for (int g0 = 0; g0 < a.groups; g0 += L) {
            const int g = g0 + sub;
            if (g < a.groups) {
                const int mine = ranks[g];
                int better = 0;
                for (int o = 0; o < a.groups; ++o) better += ranks[o] - (o >= g) >= mine;
                weigh(better < a.top_groups, g);
                if (better >= a.top_groups)
                    for (int i = 0; i < size; ++i) values[g * size + i] = kNone;
            }
        }
        wave_fence();
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (H::expert_at(r, sub) < a.experts) c[r] = values[H::expert_at(r, sub)];
    }
    wave_fence();  // the room may be written again
    if (!COMPUTED) return true;
    best = fold_max<LOG>(best);
    return best == kNone || fold_min<LOG>(worst) > best;
}

// The top_k largest choices, lane i keeping the i-th's expert, -1 where there is none.
// Equal ones in the order of their experts.
template <int LOG, int R>
__device__ __forceinline__ int largest(int top_k, int sub, int (&c)[R]) {
    typedef Held<LOG, R> H;
    int id = -1;
    for (int i = 0; i < top_k; ++i) {
        int best = kNone;
#pragma unroll
        for (int r = 0; r < R; ++r) best = max(best, c[r]);
        best = fold_max<LOG>(best);
        int at = 0x3FFFFFFF;
#pragma unroll
        for (int r = R - 1; r >= 0; --r) at = c[r] == best ? H::expert_at(r, 0) : at;
        at = best > kNone ? fold_min<LOG>(at + sub * H::V) : -1;
        const int mine = at - sub * H::V;
#pragma unroll
        for (int r = 0; r < R; ++r) c[r] = H::expert_at(r, 0) == mine ? kNone : c[r];
        if (sub == i) id = at;
    }
    return id;
}

// Keys in falling order, by comparators; of 16 only the first 8.
__device__ __forceinline__ void order(int &a, int &b) {
    const int low = min(a, b);
    a = max(a, b);
    b = low;
}
template <int O, int R>
__device__ __forceinline__ void sort8(int (&h)[R]) {
    order(h[O], h[O + 1]), order(h[O + 2], h[O + 3]), order(h[O + 4], h[O + 5]), order(h[O + 6], h[O + 7]);
    order(h[O], h[O + 2]), order(h[O + 1], h[O + 3]), order(h[O + 4], h[O + 6]), order(h[O + 5], h[O + 7]);
    order(h[O + 1], h[O + 2]), order(h[O + 5], h[O + 6]);
    order(h[O], h[O + 4]), order(h[O + 1], h[O + 5]), order(h[O + 2], h[O + 6]), order(h[O + 3], h[O + 7]);
    order(h[O + 2], h[O + 4]), order(h[O + 3], h[O + 5]);
    order(h[O + 1], h[O + 2]), order(h[O + 3], h[O + 4]), order(h[O + 5], h[O + 6]);
}
template <int R>
__device__ __forceinline__ void sort_heads(int (&k)[R]) {
    if constexpr (R == 4) {
        order(k[0], k[1]), order(k[2], k[3]), order(k[0], k[2]), order(k[1], k[3]), order(k[1], k[2]);
    } else if constexpr (R >= 8) {
        sort8<0>(k);
        if constexpr (R == 16) {
            sort8<8>(k);
            each<8>([&](auto i) { k[i] = max(k[i], k[15 - i]); });
            each<3>([&](auto s) {
                constexpr int d = 4 >> decltype(s)::value;
                each<8>([&](auto i) {
                    if constexpr (!(decltype(i)::value & d)) order(k[i], k[i + d]);
                });
            });
        }
    }
}

// The top_k largest choices by sorted lists: each lane sorts its keys once, and a step
// takes the largest head of a token's lanes, whose lane writes it down.  (Searching every
// key in every step took 1.2 of the router's 1.6 thousand instructions a wave at 65536 x
// 256, top 8; to hand each step's expert to all lanes 0.35 of them.)
//
// EXACT: keys of 16-bit logits, whose low bits hold the expert, so that they are all
// different and in the order wanted.  Otherwise the low bits hold which of the lane's
// it was, and choices that are not `gap` and the bits so lost apart may be in either order.
// lost: a choice may be missing.  room: LDS of this token, 2 L + 2 words: up to L + 1 choices, so that
// one behind the last is known where a token's lanes are all taken, and their lanes.
template <bool EXACT, int LOG, int R>
struct SortedChoice {
    typedef Held<LOG, R> H;
    static constexpr int D = R < 8 ? R : 8, LOW = EXACT ? H::L * R - 1 : R - 1, kLanes = H::L + 1;

    // Turns keys into this lane's list.
    static __device__ __forceinline__ void sort(int (&h)[R], int sub, int *room) {
        each<R>([&](auto r) {  // none: kNone or less
            h[r] = (h[r] & ~LOW) | (LOW - (EXACT ? H::expert_at(r, sub) : (int)r));
        });
        sort_heads(h);
        room[sub] = room[H::L] = kNone;
        wave_fence();
    }
    // Writes down the choices from..count - 1, count at most L + 1; popped: how many were this lane's.
    static __device__ __forceinline__ bool take(int (&h)[R], int &popped, int from, int count, int sub, int *room) {
        bool lost = false;
        for (int taken = from; taken < count; ++taken) {
            const int best = fold_max<LOG>(h[0]);
            const bool some = best > kNone, hit = some && h[0] == best;
            if (hit) {
                room[taken] = best;
                if (!EXACT) room[kLanes + taken] = sub;
            }
            if (!EXACT) {
                const uint64_t hits = __builtin_amdgcn_ballot_w64(hit), lanes = __builtin_amdgcn_ballot_w64(some);
                if (__builtin_popcountll(hits) != __builtin_popcountll(lanes) >> LOG) lost = true;  // two alike
            }
            each<D>([&](auto i) {
                int next = kNone;
                if constexpr (decltype(i)::value + 1 < D) next = h[decltype(i)::value + 1];
                const int own = h[i];
                h[i] = hit ? next : own;
            });
            popped += hit;
        }
        wave_fence();
        return lost || (D < R && popped >= D);  // this lane's list is used up, its keys may not be
    }
    static __device__ __forceinline__ float value(const int *room, int i) { return of_key(room[i] & ~LOW); }
    // Whether choices with these keys lie apart.  The low bits that hold R numbers are up to (R - 1) 2^-23
    // of the choice, its own rounding 2^-24 of it: with 16, 15.5 of the 16 2^-23 here.
    static __device__ __forceinline__ bool apart(float high, float low, float gap) {
        static_assert(EXACT || R <= 16, "the bits that keys lose");
        return high - low > gap + 0x1p-19f * (fabsf(high) + fabsf(low));
    }
    // Whether the choice after lane sub's lies apart from it, or there is none.
    static __device__ __forceinline__ bool clear(const int *room, int taken, int sub, float gap) {
        return sub + 1 >= taken || room[sub + 1] <= kNone || apart(value(room, sub), value(room, sub + 1), gap);
    }
    // Lane sub's choice, -1 where there is none.
    static __device__ __forceinline__ int expert(const int *room, int taken, int sub) {
        const int best = room[sub], low = LOW - (best & LOW);
        return sub < taken && best > kNone ? (EXACT ? low : H::expert_at(low, room[kLanes + sub])) : -1;
    }
};

// Choices of a sigmoid and a bias that lie too close together in f32: lane i has
// candidate i of `count`, which are put in the order of their 64-bit values.
template <int LOG>
__device__ __forceinline__ int order_candidates(const RouteArgs &a, int64_t row, int sub, int count, int id, double *room) {
    const double none = -(double)kInf;
    double mine = none;
    if (id >= 0 && sub < count)
        mine = 1.0 / (1.0 + exp(-(double)load_logit(a.logits, a.type, row + id))) + (double)a.bias[id];
    room[sub] = mine;
    wave_fence();
    int rank = 0;
    for (int o = 0; o < count; ++o) {
        const int e = __shfl(id, o, 1 << LOG);
        const double that = room[o];
        rank += that > mine || (that == mine && that > none && e < id);
    }
    wave_fence();
    int *const out = (int *)room;
    out[sub] = -1;
    wave_fence();
    if (mine > none) out[rank] = id;
    wave_fence();
    id = out[sub];
    wave_fence();
    return id;
}

// The same choice from 64-bit values, for waves whose f32 ones lie too close together.
// Few need it, so it takes few registers at a time, and a wave that does takes about 7 us.
// room: experts + groups values.
template <int LOG, int R>
__device__ __forceinline__ int choose_wide(const RouteArgs &a, int sub, float top, const float (&l)[R], const float (&bias)[R],
                                           double *room) {
    typedef Held<LOG, R> H;
    constexpr int L = H::L;
    const double none = -(double)kInf;
    double sum = 0.0, c[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = H::expert_at(r, sub);
        const double x = exp(a.score == LOOM_SIGMOID ? -(double)l[r] : (double)l[r] - (double)top);
        if (e < a.experts) room[e] = a.score == LOOM_SIGMOID ? 1.0 / (1.0 + x) : x;
        sum += x;
        __builtin_amdgcn_sched_barrier(0);  // one exponential after the other
    }
    sum = a.score == LOOM_SIGMOID ? 1.0 : fold_sum<LOG>(sum);
    wave_fence();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = H::expert_at(r, sub);
        if (e < a.experts) room[e] = l[r] == -kInf ? none : room[e] / sum + (double)bias[r];
        __builtin_amdgcn_sched_barrier(0);
    }
    wave_fence();
    if (a.groups > 1) {
        const int size = a.experts / a.groups;
        double *const ranks = room + a.experts;
        for (int g = sub; g < a.groups; g += L) {
            double first = none, second = none;
#pragma unroll 4
            for (int i = 0; i < size; ++i) {
                const double v = room[g * size + i], low = v < first ? v : first;
                second = low > second ? low : second;
                first = v > first ? v : first;
            }
            ranks[g] = a.group_top > 1 && second > none ? first + second : first;
        }
        wave_fence();
        for (int g = sub; g < a.groups; g += L) {
            const double mine = ranks[g];
            int better = 0;
#pragma unroll 4
            for (int o = 0; o < a.groups; ++o) better += ranks[o] > mine || (ranks[o] == mine && o < g);
            if (better >= a.top_groups)
                for (int i = 0; i < size; ++i) room[g * size + i] = none;
        }
        wave_fence();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = H::expert_at(r, sub);
        c[r] = e < a.experts ? room[e] : none;
        if (!a.bias && c[r] > none) c[r] = (double)l[r];  // the logits order the experts
    }
    int id = -1;
    for (int i = 0; i < a.top_k; ++i) {
        double best = none;
#pragma unroll
        for (int r = 0; r < R; ++r) best = c[r] > best ? c[r] : best;
        best = fold_max<LOG>(best);
        int at = 0x3FFFFFFF;
#pragma unroll
        for (int r = R - 1; r >= 0; --r) at = c[r] == best ? H::expert_at(r, 0) : at;
        at = best > none ? fold_min<LOG>(at + sub * H::V) : -1;
        const int mine = at - sub * H::V;
#pragma unroll
        for (int r = 0; r < R; ++r) c[r] = H::expert_at(r, 0) == mine ? none : c[r];
        if (sub == i) id = at;
    }
    wave_fence();
    return id;
}

// The top_k largest of the logits whose keys these are.
template <int LOG, int R>
__device__ __forceinline__ int largest_logits(const RouteArgs &a, int sub, int bad, int (&c)[R], int *room) {
    int id, h[R], popped = 0;
    bool sure;
    each<R>([&](auto r) { h[r] = c[r]; });
    if (a.type == LOOM_F32) {
        typedef SortedChoice<false, LOG, R> Sorted;
        const int taken = a.top_k + 1;
        Sorted::sort(h, sub, room);
        const bool lost = Sorted::take(h, popped, 0, taken, sub, room);
        id = Sorted::expert(room, taken, sub);
        sure = !lost && Sorted::clear(room, taken, sub, 0.0f);
    } else {
        typedef SortedChoice<true, LOG, R> Sorted;
        Sorted::sort(h, sub, room);
        sure = !Sorted::take(h, popped, 0, a.top_k, sub, room);
        id = Sorted::expert(room, a.top_k, sub);
    }
    wave_fence();
    if (__ballot(!sure && !bad)) id = largest<LOG, R>(a.top_k, sub, c);
    return id;
}

template <int LOG, int R>
__global__ __launch_bounds__(kRouteWaves * kWave, R == 16 ? (LOG == 4 ? 3 : 2) : 4) void route_kernel(RouteArgs given) {
    RouteArgs a = given;
    typedef Held<LOG, R> H;
    constexpr int L = H::L, PER = kRouteWaves * kWave / L;  // tokens of a workgroup
    int sub = threadIdx.x % L;
    const int slot = threadIdx.x / L;
    extern __shared__ char lds[];
    double *const room = (double *)lds + slot * route_room(a.experts, a.groups);
    const bool sigmoid = a.score == LOOM_SIGMOID;
    // choices, or groups' values, that are computed; else logits, which need no rounding
    const bool computed = a.bias || (a.groups > 1 && a.group_top > 1);
    float bias[R];
    bool odd = false;
#pragma unroll
    for (int r = 0; r < R; ++r) bias[r] = 0.0f;
    if (a.bias) {
        load_row<LOG, R>(a.bias, a.experts, sub, 0.0f, bias);
#pragma unroll
        for (int r = 0; r < R; ++r) odd |= bias[r] != bias[r];
    }
    const bool any_odd = __ballot(odd);
    for (int64_t base = (int64_t)blockIdx.x * PER; base < a.tokens; base += (int64_t)gridDim.x * PER) {
        const int64_t t = base + slot < a.tokens ? base + slot : a.tokens - 1;
        const int64_t row = t * a.stride;
        // what follows from these two is computed where it is used: kept over the tokens, a
        // mask for every expert a lane holds would fill the scalar registers
        asm volatile("" : "+s"(a.experts), "+v"(sub));
        float l[R];
        load_logits<LOG, R>(a.logits, a.type, row, a.experts, sub, -kInf, l);
        int bad = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) bad |= !(l[r] < kInf);
        if (any_odd) {  // a NaN bias of an expert that is not masked
#pragma unroll
            for (int r = 0; r < R; ++r) bad |= l[r] > -kInf && a.bias[H::expert_at(r, sub)] != a.bias[H::expert_at(r, sub)];
        }
        bad = fold_or<LOG>(bad);
        float top = 0.0f, total = 1.0f, s[R];
        if (!sigmoid && (computed || !a.renormalize)) {
            int highest = kNone;
#pragma unroll
            for (int r = 0; r < R; ++r) highest = max(highest, key_of(l[r]));
            highest = fold_max<LOG>(highest);
            top = highest == kNone ? 0.0f : of_key(highest);  // 0: no expert at all
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) sum += s[r] = __builtin_amdgcn_exp2f((l[r] - top) * 1.4426950408889634f);
            total = fold_sum<LOG>(sum);
        }
        int id;
        if (computed) {
            // In f32 first.  A sigmoid's error is below 2^-22 (the exponential's relative error, (1.3 |l| + 2)
            // 2^-24, counts s (1 - s) times, and |l| s (1 - s) < 0.23; the reciprocal's is 2^-23), a softmax's below
            // 2^-18 of it (31 additions, the terms' 2^-22 and a mean distance of at most 7 from the largest): two of
            // them differ by `gap`.  The sum with the bias rounds to 2^-24 of the choice, which comparisons count.
            const float unit = 1.0f / total;  // a softmax's largest score
            const float gap = sigmoid ? 0x1p-21f : unit * 0x1p-17f;
            int choice[R];
            if (sigmoid) each<R>([&](auto r) { s[r] = loom::sigmoid(l[r]); });
            else each<R>([&](auto r) { s[r] = s[r] * unit; });
            each<R>([&](auto r) {
                const int key = key_of(s[r] + bias[r]);
                choice[r] = l[r] == -kInf ? kNone : key;
            });
            bool sure = true;
            if (a.groups > 1) sure = best_groups<true, LOG, R>(a, sub, (float *)room, choice, gap);
            if (a.bias) {
                typedef SortedChoice<false, LOG, R> Sorted;
                int *const list = (int *)room, taken = a.top_k + 1;
                int popped = 0;
                Sorted::sort(choice, sub, list);
                bool lost = Sorted::take(choice, popped, 0, taken, sub, list);
                id = Sorted::expert(list, taken, sub);
                if (__ballot((lost || !Sorted::clear(list, taken, sub, gap)) && !bad)) {
                    if (sigmoid && a.top_k + 4 <= L) {
                        // three candidates more, all in the order of their 64-bit values: whoever is behind
                        // them must lie clearly behind the last choice
                        const int count = a.top_k + 4;
                        lost |= Sorted::take(choice, popped, taken, count, sub, list);
                        id = Sorted::expert(list, count, sub);
                        sure &= !lost && (list[count - 1] <= kNone ||
                                          Sorted::apart(Sorted::value(list, a.top_k - 1), Sorted::value(list, count - 1), gap));
                        wave_fence();
                        id = order_candidates<LOG>(a, row, sub, count, id, room);
                    } else {
                        sure = false;
                    }
                }
                wave_fence();
            } else {
                each<R>([&](auto r) {
                    const int key = key_of(l[r]), old = choice[r];
                    choice[r] = old == kNone ? kNone : key;
                });
                id = largest_logits<LOG, R>(a, sub, bad, choice, (int *)room);
            }
            if (__ballot(!sure && !bad)) id = choose_wide<LOG, R>(a, sub, top, l, bias, room);
        } else {
            int c[R];
#pragma unroll
            for (int r = 0; r < R; ++r) c[r] = key_of(l[r]);
            if (a.groups > 1) best_groups<false, LOG, R>(a, sub, (float *)room, c, 0.0f);
            id = largest_logits<LOG, R>(a, sub, bad, c, (int *)room);
        }
        const bool live = id >= 0 && sub < a.top_k;
        const float mine = live ? load_logit(a.logits, a.type, row + id) : 0.0f;
        float w;
        if (a.renormalize) {
            float shift;
            w = relative_score<LOG>(a.score, mine, live, shift);
            w = w / fold_sum<LOG>(w);
        } else {
            w = sigmoid ? 1.0f / (1.0f + expf(-mine)) : expf(mine - top) / total;
        }
        if (sub < a.top_k && base + slot < a.tokens) {
            a.ids[t * a.top_k + sub] = bad ? sub : id;
            a.weights[t * a.top_k + sub] = bad ? __builtin_nanf("") : live ? w * a.scale : 0.0f;
        }
    }
}

// ---------------------------------------------------------------- its gradient
// With d the gradient of the weights times scale, over the chosen experts i:
//     softmax:   d_l[j] = s_j (d_j - sum_i s_i d_i)         d_j = 0 elsewhere
//     sigmoid:   d_l[i] = d_i s_i (1 - s_i)
//     renormalised, w_i = s_i / sum s:
//                d_l[i] = w_i (d_i - sum w d), times 1 - s_i for a sigmoid
// An expert that was chosen several times takes the sum of its terms in order.
template <int LOG, int R>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_backward_kernel(RouteArgs a) {
    typedef Held<LOG, R> H;
    constexpr int L = H::L, PER = kRouteWaves * kWave / L;
    __shared__ __align__(16) float room[PER][L * R];
    const int sub = threadIdx.x % L, slot = threadIdx.x / L;
    float *const terms = room[slot];
    const bool whole = a.score == LOOM_SOFTMAX && !a.renormalize;
    for (int64_t base = (int64_t)blockIdx.x * PER; base < a.tokens; base += (int64_t)gridDim.x * PER) {
        const int64_t t = base + slot < a.tokens ? base + slot : a.tokens - 1;
        const int64_t row = t * a.stride;
        int id = sub < a.top_k ? a.ids[t * a.top_k + sub] : -1;
        if (id < 0 || id >= a.experts) id = -1;
        const bool live = id >= 0;
        const float mine = live ? load_logit(a.logits, a.type, row + id) : 0.0f;
        const float d = live ? a.d_weights[t * a.top_k + sub] * a.scale : 0.0f;
        float p[R], all = 0.0f, add;
#pragma unroll
        for (int r = 0; r < R; ++r) p[r] = 0.0f;
        if (whole) {
            load_logits<LOG, R>(a.logits, a.type, row, a.experts, sub, -kInf, p);
            float top = -kInf, sum = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) top = fmaxf(top, p[r]);
            top = fold_max<LOG>(top);
            if (top == -kInf) top = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) sum += p[r] = __builtin_amdgcn_exp2f((p[r] - top) * 1.4426950408889634f);
            sum = fold_sum<LOG>(sum);
            const float inverse = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
            const float s = live ? expf(mine - top) * inverse : 0.0f;
            add = s * d;
            all = fold_sum<LOG>(add);
#pragma unroll
            for (int r = 0; r < R; ++r) p[r] = -(p[r] * inverse) * all;
        } else if (a.renormalize) {
            float shift, w = relative_score<LOG>(a.score, mine, live, shift);
            const float sum = fold_sum<LOG>(w);
            w = sum > 0.0f || sum != sum ? w / sum : 0.0f;
            add = w * (d - fold_sum<LOG>(w * d));
            // 1 - sigmoid(l) = sigmoid(-l)
            if (a.score == LOOM_SIGMOID) add = add / (1.0f + expf(mine));
        } else {
            const float e = expf(-fabsf(mine));
            add = d * e / ((1.0f + e) * (1.0f + e));
        }
        // the chosen experts' terms meet the others through LDS; of routes with one expert
        // the first brings the sum of all in their order
        float sum = 0.0f;
        bool first = live;
        for (int i = 0; i < a.top_k; ++i) {
            const int e = __shfl(id, i, L);
            const float v = __shfl(add, i, L);
            sum += e == id ? v : 0.0f;
            first &= e != id || i >= sub;
        }
#pragma unroll
        for (int r = 0; r < R; r += H::V) *(typename H::Values *)(terms + H::expert_at(r, sub)) = typename H::Values{};
        wave_fence();
        if (first) terms[id] = sum;
        wave_fence();
#pragma unroll
        for (int r = 0; r < R; r += H::V) {
            const typename H::Values v = *(const typename H::Values *)(terms + H::expert_at(r, sub));
#pragma unroll
            for (int i = 0; i < H::V; ++i) p[r + i] += v[i];
        }
        wave_fence();
        if (base + slot < a.tokens) store_row<LOG, R>(a.d_logits, a.type, t * a.d_stride, a.experts, sub, p);
    }
}

template <int N> using Const = std::integral_constant<int, N>;
template <typename Use>
void with_lanes(int64_t tokens, int64_t experts, int64_t top_k, Use &&use) {
    const int log = route_log_lanes(tokens, experts, top_k);
    const int64_t held = route_held(tokens, experts, top_k) >> log;
    if (log == 4) {
        if (held == 4) return use(Const<4>{}, Const<4>{});
        if (held == 8) return use(Const<4>{}, Const<8>{});
        return use(Const<4>{}, Const<16>{});
    }
    if (held == 1) return use(Const<6>{}, Const<1>{});
    if (held == 4) return use(Const<6>{}, Const<4>{});
    return use(Const<6>{}, Const<16>{});
}

}  // namespace

hipError_t launch_route_experts(const loom_launch_config &cfg, const RouteArgs &a, hipStream_t stream) {
    const dim3 grid(cfg.workgroups[0]), block(cfg.workgroup_size[0]);
    with_lanes(a.tokens, a.experts, a.top_k, [&](auto log, auto held) {
        hipLaunchKernelGGL((route_kernel<decltype(log)::value, decltype(held)::value>), grid, block,
                           cfg.workgroup_storage_bytes, stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_route_experts_backward(const loom_launch_config &cfg, const RouteArgs &a, hipStream_t stream) {
    const dim3 grid(cfg.workgroups[0]), block(cfg.workgroup_size[0]);
    with_lanes(a.tokens, a.experts, a.top_k, [&](auto log, auto held) {
        hipLaunchKernelGGL((route_backward_kernel<decltype(log)::value, decltype(held)::value>), grid, block, 0, stream, a);
    });
    return hipGetLastError();
}

}  // namespace loom
