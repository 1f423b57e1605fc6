// activation.cuh -- the activations of the gated feed-forward block and their
// derivatives, in 32 bits.
#pragma once

#include "common.cuh"

namespace ddg {

// 1 / x and 2^x by one instruction each (2^-22; results below 2^-126 become 0).
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a = act(g); with D also da = act'(g).  The epilogues evaluate one for every
// accumulator while the tensor core works on the next tile, so instructions
// count: with the library's erf and tanh the products of short depth (1280)
// were bound by them.
//
// gelu: with c = erfc(|g| / sqrt 2) / 2 it is g c (g < 0) or g (1 - c).  c
// exp(g^2 / 2) falls like 1 / |g|; with t = 1 / (1 + p |g|) it is t times a
// polynomial of degree 7, fitted here for the least largest relative error over
// all g (linear programming over t in (0, 1], p chosen for it: 1.0e-6 with these
// rounded coefficients).  With the roundings in 32 bits c is good to 2^-18 down to
// g = -8 (the exponent's roundings grow as g^2): a form good to 1.5e-7 of 1 has
// 5e-4 of the result left at g = -4.  gelu_tanh: (1 + tanh z) / 2 = 1 / (1 +
// exp(-2 z)).
template <int ACT, bool D>
__device__ __forceinline__ void activation(float g, float& a, float& da) {
    if (ACT == DDGEMM_ACT_SILU) {
        const float s = __fdividef(1.0f, 1.0f + __expf(-g));  // 0 where exp overflows
        a = g * s;
        if (D) da = s * (1.0f + g * (1.0f - s));
    } else if (ACT == DDGEMM_ACT_GELU) {
        const float t = reciprocal(fmaf(0.326f, fabsf(g), 1.0f)), e = exp2_approx(g * g * -0.72134752044448170f);  // log2(e) / 2
        float q = fmaf(t, 0.0337685347f, -0.112105384f);
        q = fmaf(t, q, 0.0818242058f);
        q = fmaf(t, q, 0.0275431797f);
        q = fmaf(t, q, 0.0929912031f);
        q = fmaf(t, q, 0.115857609f);
        q = fmaf(t, q, 0.130065829f);
        q = fmaf(t, q, 0.130055189f);
        q = q * t * e;  // erfc(|g| / sqrt 2) / 2
        const float c = g < 0.0f ? q : 1.0f - q;
        a = g * c;
        if (D) da = fmaf(g * 0.39894228040143268f, e, c);
    } else if (ACT == DDGEMM_ACT_GELU_TANH) {
        const float k2 = 1.59576912160573072f, r = 0.044715f;  // 2 sqrt(2 / pi)
        const float gg = fminf(g * g, 1e6f);  // the sigmoid is 0 or 1 long before
        const float s = __fdividef(1.0f, 1.0f + __expf(-k2 * g * fmaf(r, gg, 1.0f)));
        a = g * s;
        if (D) da = s * fmaf(g * (1.0f - s), k2 * fmaf(3.0f * r, gg, 1.0f), 1.0f);
    } else {
        a = fmaxf(g, 0.0f);
        if (g != g) a = g;  // NaN stays NaN
        if (D) da = g > 0.0f ? 1.0f : 0.0f;
    }
}

// Calls f(std::integral_constant<int, act>) for the activation chosen at run
// time, so that the choice is made once per tile and not per element.
template <int V> struct ActTag { static constexpr int value = V; };
template <class F>
__device__ __forceinline__ void with_activation(int act, F f) {
    switch (act) {
        case DDGEMM_ACT_SILU: f(ActTag<DDGEMM_ACT_SILU>{}); break;
        case DDGEMM_ACT_GELU: f(ActTag<DDGEMM_ACT_GELU>{}); break;
        case DDGEMM_ACT_GELU_TANH: f(ActTag<DDGEMM_ACT_GELU_TANH>{}); break;
        default: f(ActTag<DDGEMM_ACT_RELU>{}); break;
    }
}

}  // namespace ddg
