// The gates of the gated blocks: a(g), its slope, the limit on g and u, and
// the choice among them.
//
// Every function of g passes a NaN on, and the limits are comparisons that a NaN
// fails for the same reason (fmin would drop it).
#pragma once

#include <type_traits>

#include "philox.h"

namespace moe {

// g' = min(g, L), u' = clamp(u, -L, L); no limit: L = infinity
__device__ __forceinline__ float limit_g(float g, float L) { return g > L ? L : g; }
__device__ __forceinline__ float limit_u(float u, float L) { return u > L ? L : (u < -L ? -L : u); }

// the same, or nothing where it is known that there is no limit (LIM false): the gradient through relu of 32768 rows
// takes 467 us with the comparisons, 451 without
template <bool LIM>
struct Limit {
    float L;
    __device__ __forceinline__ float g(float v) const { return LIM ? limit_g(v, L) : v; }
    __device__ __forceinline__ float u(float v) const { return LIM ? limit_u(v, L) : v; }
    __device__ __forceinline__ float slope_g(float v, float d) const { return LIM && v > L ? 0.0f : d; }
    __device__ __forceinline__ float slope_u(float v, float d) const { return LIM && (v > L || v < -L) ? 0.0f : d; }
};

// 1 / (1 + exp(-z)).  FAST: the hardware's exp2 and reciprocal (bf16 results:
// their 2^-22 is far below the rounding), else the library's.
template <bool FAST>
__device__ __forceinline__ float sigmoid_of(float z)
{
    if constexpr (FAST) return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    else return 1.0f / (1.0f + expf(-z));
}

// Phi(g) and exp(-g^2 / 2) for the erf form of GELU.  FAST: erfc(x) =
// exp(-x^2) t P(t) with t = 1 / (1 + 0.375 x) for x >= 0, P a polynomial of
// degree 6 fitted to the relative error (1e-6 over [0, 12], beyond which exp
// is 0), so that the tail below -3 keeps its digits; Phi(-g) = 1 - Phi(g).
// In fp32, where x^2 is rounded before exp, the tail's relative error is 4e-6
// at g = -6 and 1.6e-5 from -12 on: bf16 results round by 4e-3.
template <bool FAST>
__device__ __forceinline__ void normal_of(float g, float& Phi, float& ex)
{
    if constexpr (FAST) {
        const float x = fabsf(g) * 0.70710678f;
        ex = __expf(-x * x);
        const float t = __builtin_amdgcn_rcpf(fmaf(0.375f, x, 1.0f));
        float q = -0.133232538f;
        q = fmaf(q, t, 0.381480544f);
        q = fmaf(q, t, -0.120656477f);
        q = fmaf(q, t, 0.276759115f);
        q = fmaf(q, t, 0.169039063f);
        q = fmaf(q, t, 0.215237705f);
        q = fmaf(q, t, 0.211373188f);
        const float half = 0.5f * ex * t * q;      // Phi(-|g|)
        Phi = g < 0.0f ? half : 1.0f - half;
    } else {
        ex = expf(-0.5f * g * g);
        Phi = 0.5f * erfcf(g * -0.70710678118654752f);
    }
}

// the tanh form's s = sigmoid(z) with z = 2 sqrt(2/pi) (g + 0.044715 g^3), and
// dz/dg.  Past |g| = 12 s is 0 or 1 in fp32 (z = 142), so g^3 is formed from
// g held there: no infinity meets a zero.  (A NaN is lost here and kept by
// the products with g itself.)
template <bool FAST>
__device__ __forceinline__ float gelu_tanh_sigmoid(float g, float& dz)
{
    const float c = __builtin_amdgcn_fmed3f(g, -12.0f, 12.0f);
    const float c2 = c * c;
    dz = fmaf(0.2140644481f, c2, 1.5957691216f);               // 2 sqrt(2/pi) (1 + 3 * 0.044715 g^2)
    return sigmoid_of<FAST>(c * fmaf(0.0713548160f, c2, 1.5957691216f));
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_of(float g)
{
    if constexpr (ACT == MOE_ACT_SILU) {
        return g * sigmoid_of<FAST>(g);
    } else if constexpr (ACT == MOE_ACT_GELU) {
        float Phi, ex;
        normal_of<FAST>(g, Phi, ex);
        return g * Phi;
    } else if constexpr (ACT == MOE_ACT_GELU_TANH) {
        float dz;
        return g * gelu_tanh_sigmoid<FAST>(g, dz);
    } else {
        return g < 0.0f ? 0.0f : g;
    }
}

// a(g) and a'(g)
template <int ACT, bool FAST>
__device__ __forceinline__ void act_and_slope(float g, float& a, float& slope)
{
    if constexpr (ACT == MOE_ACT_SILU) {
        const float s = sigmoid_of<FAST>(g);
        a = g * s;
        slope = s * fmaf(g, 1.0f - s, 1.0f);
    } else if constexpr (ACT == MOE_ACT_GELU) {
        float Phi, ex;
        normal_of<FAST>(g, Phi, ex);
        a = g * Phi;
        slope = fmaf(g * 0.39894228f, ex, Phi);
    } else if constexpr (ACT == MOE_ACT_GELU_TANH) {
        float dz;
        const float s = gelu_tanh_sigmoid<FAST>(g, dz);
        a = g * s;
        slope = s * fmaf(g * (1.0f - s), dz, 1.0f);
    } else {
        a = g < 0.0f ? 0.0f : g;
        slope = g > 0.0f ? 1.0f : 0.0f;
    }
}

// f(integral_constant<int, act>) (act checked on the host)
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f)
{
    switch (act) {
    case MOE_ACT_SILU: f(std::integral_constant<int, MOE_ACT_SILU>{}); break;
    case MOE_ACT_GELU: f(std::integral_constant<int, MOE_ACT_GELU>{}); break;
    case MOE_ACT_GELU_TANH: f(std::integral_constant<int, MOE_ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, MOE_ACT_RELU>{}); break;
    }
}

// f(integral_constant<int, act>, Limit)
template <class F>
__device__ __forceinline__ void with_glu(const GluSpec& glu, F&& f)
{
    with_act(glu.act, [&](auto A) __attribute__((always_inline)) {
        if (glu.limit < __builtin_inff()) f(A, Limit<true>{glu.limit});
        else f(A, Limit<false>{glu.limit});
    });
}

}  // namespace moe
