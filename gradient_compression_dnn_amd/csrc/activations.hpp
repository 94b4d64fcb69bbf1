// Activations, and rows of activations, as the layer products use them.
#pragma once

#include "gc_internal.hpp"

namespace gc {

// ------------------------------------------------------------- activations
// kFast: for results that are rounded to 16 bits.  The hardware's exp2 and
// reciprocal (each within a step) in place of the library's, and for Phi a
// polynomial.  A value is off by 2^-14 of itself at most, a 64th of bf16's own
// rounding; inside +-6, all that fp16 has of GELU's tail, by 2^-15, a 16th of
// its rounding.  Far out most of that is the rounding of the exponent.
template <bool kFast>
__device__ __forceinline__ float exp_of(float x) {
    return kFast ? __builtin_amdgcn_exp2f(x * 1.44269504f) : expf(x);
}
template <bool kFast>
__device__ __forceinline__ float sigmoid(float v) {
    const float d = 1.0f + exp_of<kFast>(-v);
    return kFast ? __builtin_amdgcn_rcpf(d) : 1.0f / d;
}
// And 1 - s, from the exponential where s is near 1: as a difference it loses what a factor z times it shows (fp32,
// GELU_TANH's slope off by 2.1e-7 where the difference gave 2.0e-6, SILU's 2.1e-7 and 9.8e-7).
template <bool kFast>
__device__ __forceinline__ float sigmoid(float v, float &rest) {
    const float e = exp_of<kFast>(-v), d = 1.0f + e;
    const float s = kFast ? __builtin_amdgcn_rcpf(d) : 1.0f / d;
    rest = v > 0.0f ? e * s : 1.0f - s;
    return s;
}

constexpr float kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;
// Phi(z), and e = exp(-z^2 / 2).  For kFast Phi(-a) = e g(a) with g(a) = exp(a^2 / 2) Phi(-a), which falls from
// 1/2 like 1 / a: t P(t) with t = 1 / (1 + 0.302 a) and P of degree 5, a weighted least-maximum fit of the relative
// error over 0 to 13.5, where e leaves the floats: 8.4e-6 of g, and 5.3e-7 of 1 in Phi.  A polynomial with an
// absolute bound of the same cost but one multiplication was off by 1% of itself at -8.
template <bool kFast>
__device__ __forceinline__ float normal(float z, float &e) {
    e = exp_of<kFast>(-0.5f * z * z);
    if (!kFast) return 0.5f * erfcf(-z * kSqrtHalf);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.302f, fabsf(z), 1.0f));
    float q = __builtin_fmaf(-0.0784434161f, t, 0.213962695f);
    q = __builtin_fmaf(q, t, -0.0153387377f);
    q = __builtin_fmaf(q, t, 0.144378609f);
    q = __builtin_fmaf(q, t, 0.114566279f);
    q = __builtin_fmaf(q, t, 0.120874168f);
    q = q * t * e;  // Phi(-|z|)
    return z < 0.0f ? q : 1.0f - q;
}

// 2 sqrt(2 / pi) (z + 0.044715 z^3), whose sigmoid is gelu_tanh's factor
constexpr float kTanh2 = 1.5957691216057308f, kCubic = 0.044715f;
__device__ __forceinline__ float tanh_argument(float z) { return kTanh2 * __builtin_fmaf(kCubic * z * z, z, z); }

// v = act(v)
template <bool kFast, int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    float e;
    switch (act) {
        case GC_ACT_RELU:
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = v[u] < 0.0f ? 0.0f : v[u];
            break;
        case GC_ACT_GELU:
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = v[u] * normal<kFast>(v[u], e);
            break;
        case GC_ACT_GELU_TANH:
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = v[u] * sigmoid<kFast>(tanh_argument(v[u]));
            break;
        case GC_ACT_SILU:
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = v[u] * sigmoid<kFast>(v[u]);
            break;
        default: break;
    }
}

// v = act'(v).  Beyond +-kFar every slope is 0 or 1 in fp32, and z^2 could overflow.
constexpr float kFar = 128.0f;
template <bool kFast, int N>
__device__ __forceinline__ void act_slopes(int act, float (&v)[N]) {
    switch (act) {
        case GC_ACT_RELU:
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = v[u] > 0.0f ? 1.0f : 0.0f;
            break;
        case GC_ACT_GELU:
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const float z = v[u];
                float e;
                const float p = normal<kFast>(z, e);
                v[u] = fabsf(z) > kFar ? (z > 0.0f ? 1.0f : 0.0f) : __builtin_fmaf(z * kInvSqrt2Pi, e, p);
            }
            break;
        case GC_ACT_GELU_TANH:
#pragma unroll
            for (int u = 0; u < N; ++u) {
                float rest;
                const float z = v[u], s = sigmoid<kFast>(tanh_argument(z), rest);
                const float d = kTanh2 * __builtin_fmaf(3.0f * kCubic * z, z, 1.0f);
                v[u] = fabsf(z) > kFar ? (z > 0.0f ? 1.0f : 0.0f) : __builtin_fmaf(z * (s * rest), d, s);
            }
            break;
        case GC_ACT_SILU:
#pragma unroll
            for (int u = 0; u < N; ++u) {
                float rest;
                const float z = v[u], s = sigmoid<kFast>(z, rest);
                v[u] = fabsf(z) > kFar ? (z > 0.0f ? 1.0f : 0.0f) : s * __builtin_fmaf(z, rest, 1.0f);
            }
            break;
        default:
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = 1.0f;
    }
}

// ------------------------------------------------------------------- rows
// N columns of a row as they stand in memory, of which `cnt` exist: 16 bytes at
// a time where all do.
template <class T, int N>
struct Cols {
    using Store = typename T::Store;
    static constexpr int kVec = N * int(sizeof(Store)) <= 16 ? N : 16 / int(sizeof(Store));
    Pack<Store, kVec> v[N / kVec];
    __device__ __forceinline__ void load(const void *base, uint64_t at, uint32_t cnt) {
        const Store *p = static_cast<const Store *>(base) + at;
        if (cnt >= N) {
#pragma unroll
            for (int k = 0; k < N / kVec; ++k) v[k] = *reinterpret_cast<const Pack<Store, kVec> *>(p + k * kVec);
            return;
        }
#pragma unroll
        for (uint32_t u = 0; u < N; ++u) v[u / kVec].v[u % kVec] = u < cnt ? p[u] : Store(0);
    }
    __device__ __forceinline__ float at(int u) const { return T::to_f32(v[u / kVec].v[u % kVec]); }
};
template <class T>
struct Cols<T, 0> {};

template <class T, int N>
__device__ __forceinline__ void put_cols(void *base, uint64_t at, uint32_t cnt, const float (&v)[N]) {
    using Store = typename T::Store;
    constexpr int kVec = N * int(sizeof(Store)) <= 16 ? N : 16 / int(sizeof(Store));
    Store *p = static_cast<Store *>(base) + at;
    if (cnt >= N) {
#pragma unroll
        for (int k = 0; k < N; k += kVec) {
            Pack<Store, kVec> t;
#pragma unroll
            for (int u = 0; u < kVec; ++u) t.v[u] = T::from_f32(v[k + u]);
            *reinterpret_cast<Pack<Store, kVec> *>(p + k) = t;
        }
        return;
    }
#pragma unroll
    for (uint32_t u = 0; u < N; ++u)
        if (u < cnt) p[u] = T::from_f32(v[u]);
}

}  // namespace gc
