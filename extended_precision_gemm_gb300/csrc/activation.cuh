// activation.cuh -- the activations of the gated feed-forward block and their
// derivatives, in 32 bits.
#pragma once

#include "common.cuh"

namespace ddg {

// a = act(g); with D also da = act'(g).  The epilogues evaluate one for every
// accumulator while the tensor core works on the next tile, so instructions
// count: with the library's erf and tanh the products of short depth (1280)
// were bound by them.
//
// gelu: erfc(x) = t (a1 + t (a2 + ...)) exp(-x^2), t = 1 / (1 + p x), x >= 0
// (Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26, error at
// most 1.5e-7).  gelu_tanh: (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)).
template <int ACT, bool D>
__device__ __forceinline__ void activation(float g, float& a, float& da) {
    if (ACT == DDGEMM_ACT_SILU) {
        const float s = __fdividef(1.0f, 1.0f + __expf(-g));  // 0 where exp overflows
        a = g * s;
        if (D) da = s * (1.0f + g * (1.0f - s));
    } else if (ACT == DDGEMM_ACT_GELU) {
        const float x = fabsf(g) * 0.70710678118654752f;
        const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f)), e = __expf(-x * x);
        float q = fmaf(t, 1.061405429f, -1.453152027f);
        q = fmaf(t, q, 1.421413741f);
        q = fmaf(t, q, -0.284496736f);
        q = fmaf(t, q, 0.254829592f);
        q = 0.5f * q * t * e;  // half of erfc(|g| / sqrt 2)
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
