// route_experts.hip -- routing of tokens to experts, and its gradient.
//
//     s = softmax(l) or sigmoid(l),   c = s + bias, or l itself without a bias
//     a group's value: the sum of its group_top largest c (without a bias: of s)
//     ids: the top_k largest c of the top_groups best groups, in falling order
//     w = s[ids], divided by their sum where renormalised, times scale
//
// Ties go to the lower index.  Neighbouring choices may differ by less than a
// step of f32, so wherever a choice is computed (and is not a logit itself) it
// is computed and compared in 64 bits; weights are f32.
#include <type_traits>

#include "ffn_common.hpp"

namespace loom {

namespace {

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
// 2^LOG lanes hold a token, lane i the experts i, i + 2^LOG, ..: R of them.
template <typename C, int LOG, int R>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_kernel(RouteArgs a) {
    constexpr int L = 1 << LOG, PER = kRouteWaves * kWave / L;  // tokens of a workgroup
    const int sub = threadIdx.x % L, slot = threadIdx.x / L;
    extern __shared__ char lds[];
    C *values = (C *)lds + (int64_t)slot * (a.groups > 1 ? a.experts : 0);
    C *ranks = (C *)lds + (int64_t)PER * a.experts + slot * (a.groups > 1 ? a.groups : 0);
    for (int64_t base = (int64_t)blockIdx.x * PER; base < a.tokens; base += (int64_t)gridDim.x * PER) {
        const int64_t t = base + slot < a.tokens ? base + slot : a.tokens - 1;
        const int64_t row = t * a.stride;
        float l[R], top = -kInf;
        int bad = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = r * L + sub;
            l[r] = e < a.experts ? load_logit(a.logits, a.type, row + e) : -kInf;
            bad |= !(l[r] < kInf);
            top = fmaxf(top, l[r]);
        }
        C c[R];
        float total = 1.0f;
        top = fold_max<LOG>(top);
        const float from = top == -kInf ? 0.0f : top;  // no expert at all
        if (a.score == LOOM_SOFTMAX) {
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) sum += expf(l[r] - from);
            total = fold_sum<LOG>(sum);
        }
        // the choices: computed ones are 64-bit throughout
        if constexpr (sizeof(C) == 8) {
            double sum = 0.0;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                c[r] = a.score == LOOM_SIGMOID ? 1.0 / (1.0 + exp(-(double)l[r])) : exp((double)l[r] - (double)from);
                if (a.score == LOOM_SOFTMAX) sum += c[r];
            }
            if (a.score == LOOM_SOFTMAX) sum = fold_sum<LOG>(sum);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int e = r * L + sub;
                if (a.score == LOOM_SOFTMAX) c[r] = c[r] / sum;
                if (a.bias && e < a.experts) c[r] = c[r] + (double)a.bias[e];
                bad |= e < a.experts && l[r] > -kInf && c[r] != c[r];
                if (l[r] == -kInf) c[r] = -kInf;
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) c[r] = l[r];
        }
        bad = fold_or<LOG>(bad);
        if (a.groups > 1) {
            // a lane a group: its largest values, and whether it is among the best
            const int size = a.experts / a.groups;
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r * L + sub < a.experts) values[r * L + sub] = c[r];
            __syncthreads();
            for (int g = sub; g < a.groups; g += L) {
                C first = -kInf, second = -kInf;
                for (int i = 0; i < size; ++i) {
                    const C v = values[g * size + i];
                    if (v > first) second = first, first = v;
                    else if (v > second) second = v;
                }
                ranks[g] = a.group_top > 1 && second > -kInf ? first + second : first;
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int g = (r * L + sub) / size;
                if (r * L + sub >= a.experts) continue;
                const C mine = ranks[g];
                int better = 0;
                for (int o = 0; o < a.groups; ++o) better += ranks[o] > mine || (ranks[o] == mine && o < g);
                if (better >= a.top_groups) c[r] = -kInf;
                // without a bias the logits order a group's experts
                else if (!a.bias) c[r] = l[r];
            }
        }
        int id = -1;
        for (int i = 0; i < a.top_k; ++i) {
            C best = -kInf;
#pragma unroll
            for (int r = 0; r < R; ++r) best = c[r] > best ? c[r] : best;
            best = fold_max<LOG>(best);
            int at = 0x7FFFFFFF;
#pragma unroll
            for (int r = R - 1; r >= 0; --r)
                if (c[r] == best) at = r * L + sub;
            at = fold_min<LOG>(at);
            if (!(best > -kInf)) at = -1;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r * L + sub == at) c[r] = -kInf;
            if (sub == i) id = at;
        }
        const bool live = id >= 0 && sub < a.top_k;
        const float mine = live ? load_logit(a.logits, a.type, row + id) : 0.0f;
        float w;
        if (a.renormalize) {
            float shift;
            w = relative_score<LOG>(a.score, mine, live, shift);
            w = w / fold_sum<LOG>(w);
        } else {
            w = a.score == LOOM_SIGMOID ? 1.0f / (1.0f + expf(-mine)) : expf(mine - from) / total;
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
    constexpr int L = 1 << LOG, PER = kRouteWaves * kWave / L;
    const int sub = threadIdx.x % L, slot = threadIdx.x / L;
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
            float top = -kInf, sum = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int e = r * L + sub;
                p[r] = e < a.experts ? load_logit(a.logits, a.type, row + e) : -kInf;
                top = fmaxf(top, p[r]);
            }
            top = fold_max<LOG>(top);
            if (top == -kInf) top = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                p[r] = expf(p[r] - top);
                sum += p[r];
            }
            sum = fold_sum<LOG>(sum);
            const float inverse = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) p[r] = p[r] * inverse;
            const float s = live ? expf(mine - top) * inverse : 0.0f;
            all = fold_sum<LOG>(s * d);
            add = s * d;
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
        float out[R];
#pragma unroll
        for (int r = 0; r < R; ++r) out[r] = whole ? -p[r] * all : 0.0f;
        for (int i = 0; i < a.top_k; ++i) {
            const int e = __shfl(id, i, L);
            const float v = __shfl(add, i, L);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r * L + sub == e) out[r] += v;
        }
        if (base + slot < a.tokens) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r * L + sub < a.experts) store1(a.d_logits, a.type, t * a.d_stride + r * L + sub, out[r]);
        }
    }
}

template <int N> using Const = std::integral_constant<int, N>;
template <typename Use>
void with_lanes(int64_t tokens, int64_t experts, int64_t top_k, Use &&use) {
    const int log = route_log_lanes(tokens, experts, top_k);
    const int held = (int)((experts + (1 << log) - 1) >> log);
    if (log == 4) {
        if (held <= 4) return use(Const<4>{}, Const<4>{});
        if (held <= 8) return use(Const<4>{}, Const<8>{});
        return use(Const<4>{}, Const<16>{});
    }
    if (held <= 1) return use(Const<6>{}, Const<1>{});
    if (held <= 4) return use(Const<6>{}, Const<4>{});
    return use(Const<6>{}, Const<16>{});
}

}  // namespace

hipError_t launch_route_experts(const loom_launch_config &cfg, const RouteArgs &a, hipStream_t stream) {
    const dim3 grid(cfg.workgroups[0]), block(cfg.workgroup_size[0]);
    with_lanes(a.tokens, a.experts, a.top_k, [&](auto log, auto held) {
        constexpr int LOG = decltype(log)::value, R = decltype(held)::value;
        if (a.bias || (a.groups > 1 && a.group_top > 1))
            hipLaunchKernelGGL((route_kernel<double, LOG, R>), grid, block, cfg.workgroup_storage_bytes, stream, a);
        else
            hipLaunchKernelGGL((route_kernel<float, LOG, R>), grid, block, cfg.workgroup_storage_bytes, stream, a);
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
