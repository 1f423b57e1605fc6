// activation.cuh -- the activations of the gated feed-forward block and their
// derivatives, in 32 bits.
#pragma once

#include "common.cuh"

namespace ddg {

// a = act(g); with D also da = act'(g).
template <int ACT, bool D>
__device__ __forceinline__ void activation(float g, float& a, float& da) {
    if (ACT == DDGEMM_ACT_SILU) {
        const float s = __fdividef(1.0f, 1.0f + __expf(-g));  // 0 where exp overflows
        a = g * s;
        if (D) da = s * (1.0f + g * (1.0f - s));
    } else if (ACT == DDGEMM_ACT_GELU) {
        const float c = 0.5f * (1.0f + erff(g * 0.70710678118654752f));
        a = g * c;
        if (D) da = c + g * (0.39894228040143268f * __expf(-0.5f * g * g));
    } else if (ACT == DDGEMM_ACT_GELU_TANH) {
        const float k = 0.79788456080286536f, q = 0.044715f;
        const float t = tanhf(k * g * (1.0f + q * g * g));
        a = 0.5f * g * (1.0f + t);
        if (D) da = 0.5f * (1.0f + t) + 0.5f * g * (1.0f - t * t) * k * (1.0f + 3.0f * q * g * g);
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
