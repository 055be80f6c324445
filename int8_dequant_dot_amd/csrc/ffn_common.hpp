// ffn_common.hpp -- element types and activations shared by the int8
// feed-forward kernels (row quantiser, product, gated projection, gradients).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "internal.hpp"

namespace loom {

template <int TYPE> struct ElementOf;
template <> struct ElementOf<LOOM_F32> { typedef float type; };
template <> struct ElementOf<LOOM_F16> { typedef _Float16 type; };
template <> struct ElementOf<LOOM_BF16> { typedef __bf16 type; };

__host__ __device__ __forceinline__ constexpr int element_bytes(int type) { return type == LOOM_F32 ? 4 : 2; }

// One value, or four neighbours (one store where `whole` says the row allows
// it, or the first `left`), rounded once to the output type; the branch on the
// type is the same in every lane.
template <typename T>
__device__ __forceinline__ void store4_as(T *to, int64_t left, bool whole, const float (&y)[4]) {
    typedef T V __attribute__((ext_vector_type(4)));
    if (whole && left >= 4) {
        *(V *)to = V{(T)y[0], (T)y[1], (T)y[2], (T)y[3]};
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < left) to[e] = (T)y[e];
}
__device__ __forceinline__ void store4(void *out, int type, int64_t at, int64_t left, bool whole,
                                       const float (&y)[4]) {
    if (type == LOOM_F32) store4_as((float *)out + at, left, whole, y);
    else if (type == LOOM_F16) store4_as((_Float16 *)out + at, left, whole, y);
    else store4_as((__bf16 *)out + at, left, whole, y);
}
// Four neighbours of each of N places `by` elements apart, where live: one branch
// on the type and on the row's alignment for all of them.
template <typename T, int N>
__device__ __forceinline__ void store4_each_as(T *to, int64_t by, int64_t left, bool whole, const bool (&live)[N],
                                               const float (&y)[N][4]) {
    if (whole && left >= 4) {
        typedef T V __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (live[j]) *(V *)(to + j * by) = V{(T)y[j][0], (T)y[j][1], (T)y[j][2], (T)y[j][3]};
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (live[j] && e < left) to[j * by + e] = (T)y[j][e];
    }
}
template <int N>
__device__ __forceinline__ void store4_each(void *out, int type, int64_t at, int64_t by, int64_t left, bool whole,
                                            const bool (&live)[N], const float (&y)[N][4]) {
    if (type == LOOM_F32) store4_each_as((float *)out + at, by, left, whole, live, y);
    else if (type == LOOM_F16) store4_each_as((_Float16 *)out + at, by, left, whole, live, y);
    else store4_each_as((__bf16 *)out + at, by, left, whole, live, y);
}
template <typename T>
__device__ __forceinline__ void load4_as(const T *from, int64_t left, bool whole, float (&y)[4]) {
    typedef T V __attribute__((ext_vector_type(4)));
    if (whole && left >= 4) {
        const V v = *(const V *)from;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = (float)v[e];
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = e < left ? (float)from[e] : 0.0f;
}
// Four neighbours, 0 past the first `left`.
__device__ __forceinline__ void load4(const void *in, int type, int64_t at, int64_t left, bool whole,
                                      float (&y)[4]) {
    if (type == LOOM_F32) load4_as((const float *)in + at, left, whole, y);
    else if (type == LOOM_F16) load4_as((const _Float16 *)in + at, left, whole, y);
    else load4_as((const __bf16 *)in + at, left, whole, y);
}
__device__ __forceinline__ void store1(void *out, int type, int64_t at, float y) {
    if (type == LOOM_F32) ((float *)out)[at] = y;
    else if (type == LOOM_F16) ((_Float16 *)out)[at] = (_Float16)y;
    else ((__bf16 *)out)[at] = (__bf16)y;
}

// Phi(g), the normal distribution's integral: erfc keeps the lower tail's
// relative accuracy, which 1 + erf loses.
__device__ __forceinline__ float normal_cdf(float g) { return 0.5f * erfcf(g * -0.70710678118654752f); }

// 1 / (1 + exp(-z)) with the exponential and the reciprocal of the hardware,
// each within one unit in the last place; the exponent -z log2(e) carries the
// product's rounding and the constant's (0.23 of half a step more), an error of
// 1.23 |z| 2^-24 of the exponential.  (The library's expf and a rounded quotient
// took 40 instructions, 8 % of a 4096-token projection.)
// exp overflows to infinity for z < -128 ln 2, where the result is 0.
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

// The tanh form's factor 0.5 (1 + tanh z), z = sqrt(2/pi) (g + 0.044715 g^3),
// is sigmoid(2 z).  It is 0 or 1 to f32 well inside |g| = 16, where g is held
// so that its powers stay finite; a NaN passes.
__device__ __forceinline__ float tanh_form_gate(float g) { return g > 16.0f ? 16.0f : g < -16.0f ? -16.0f : g; }
__device__ __forceinline__ float tanh_form_cdf(float c) {
    return sigmoid(1.5957691216057308f * (c + 0.044715f * c * c * c));
}

// act(g) of a gated unit.  A NaN stays a NaN in each of them.
__device__ __forceinline__ float act_value(int act, float g) {
    switch (act) {
        case LOOM_SILU: return g * sigmoid(g);
        case LOOM_GELU: return g * normal_cdf(g);
        case LOOM_GELU_TANH: return g * tanh_form_cdf(tanh_form_gate(g));
        default: return g < 0.0f ? 0.0f : g;
    }
}

// body with the activation as a compile-time constant: one branch for all that
// body computes.
template <int ACT> struct Activation { static constexpr int value = ACT; };
template <typename Body>
__device__ __forceinline__ void with_activation(int act, Body &&body) {
    switch (act) {
        case LOOM_SILU: return body(Activation<LOOM_SILU>{});
        case LOOM_GELU: return body(Activation<LOOM_GELU>{});
        case LOOM_GELU_TANH: return body(Activation<LOOM_GELU_TANH>{});
        default: return body(Activation<LOOM_RELU>{});
    }
}

// act(g) and its derivative.  ReLU's derivative at 0 is 0.
__device__ __forceinline__ void act_value_slope(int act, float g, float &value, float &slope) {
    switch (act) {
        case LOOM_SILU: {
            const float p = sigmoid(g);
            value = g * p;
            slope = p * (1.0f + g * (1.0f - p));
            return;
        }
        case LOOM_GELU: {
            const float p = normal_cdf(g);
            value = g * p;
            slope = p + g * __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f) * 0.39894228040143268f;
            return;
        }
        case LOOM_GELU_TANH: {
            const float c = tanh_form_gate(g), p = tanh_form_cdf(c);
            value = g * p;
            slope = p + c * p * (1.0f - p) * 1.5957691216057308f * (1.0f + 0.134145f * c * c);
            return;
        }
        default:
            value = g < 0.0f ? 0.0f : g;
            slope = g > 0.0f ? 1.0f : g != g ? g : 0.0f;
    }
}

}  // namespace loom
