// activation.hpp -- the gate activations of a gated feed-forward block, act(g), and their derivatives,
// in binary32 on the device.
//
//   silu       act(g) = g s(g),         s(z) = 1 / (1 + e^-z)
//   gelu       act(g) = g P(g),         P(g) = erfc(-g / sqrt 2) / 2
//   gelu_tanh  act(g) = g s(z(g)),      z(g) = sqrt(8/pi) (g + 0.044715 g^3)
//
// (0.5 (1 + tanh y) = s(2 y), so the last is the usual tanh form.)  Each keeps its relative accuracy where
// act(g) is tiny (g far below zero).
#pragma once

#include "device_common.hpp"

namespace bsq {

// act and d act / d g.
struct ActGrad {
    float f, df;
};

// e^x as the square of e^(x/2): the hardware's exp2 returns 0 for results below 2^-126, the product does not.
__device__ __forceinline__ float exp_fast(float x) {
    const float h = __builtin_amdgcn_exp2f(x * 0.721347520f);
    return h * h;
}

// s(z), from e^-|z| so that nothing overflows; a NaN passes through.
__device__ __forceinline__ float sigmoid(float z) {
    const float e = exp_fast(-__builtin_fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e);
    return z >= 0.0f ? r : e * r;
}

// P(g) = erfc(-g / sqrt 2) / 2, the normal distribution function.  With x = |g| / sqrt 2 and t = 1 / (1 +
// x / 2), erfc(x) = t e^(-x^2) Q(t) for a smooth positive Q on (0, 1]; Q's polynomial is a Chebyshev fit
// made for this file over t in [0.17, 1] (x <= 9.7, below which e^(-x^2) leaves binary32's range); its
// relative error in binary32 is 2.1e-7.
__device__ __forceinline__ float normal_cdf(float g) {
    const float x = __builtin_fabsf(g) * 0.707106781f;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, x, 1.0f));
    float q = -0.060039805f;
    q = __builtin_fmaf(q, t, 0.289117624f);
    q = __builtin_fmaf(q, t, -0.496166757f);
    q = __builtin_fmaf(q, t, 0.287778320f);
    q = __builtin_fmaf(q, t, -0.032907345f);
    q = __builtin_fmaf(q, t, 0.205159566f);
    q = __builtin_fmaf(q, t, 0.242528244f);
    q = __builtin_fmaf(q, t, 0.282447393f);
    q = __builtin_fmaf(q, t, 0.282082710f);
    const float half = 0.5f * t * q * exp_fast(-x * x);   // erfc(x) / 2
    return g >= 0.0f ? 1.0f - half : (g < 0.0f ? half : g);
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    if constexpr (ACT == 1) return g * normal_cdf(g);
    float z = g;
    if constexpr (ACT == 2) z = 1.59576912f * __builtin_fmaf(0.044715f * g * g, g, g);
    return g * sigmoid(z);
}

template <int ACT>
__device__ __forceinline__ ActGrad act_grad(float g) {
    if constexpr (ACT == 1) {
        const float p = normal_cdf(g);
        return {g * p, __builtin_fmaf(g * 0.39894228f, exp_fast(-0.5f * g * g), p)};
    }
    float z = g, dz = 1.0f;
    if constexpr (ACT == 2) {
        z = 1.59576912f * __builtin_fmaf(0.044715f * g * g, g, g);
        // kept finite, so that it stays without effect where s (1 - s) is 0
        dz = __builtin_fminf(1.59576912f * __builtin_fmaf(0.134145f * g, g, 1.0f), 3.0e38f);
    }
    // act'(g) = s + g s s(-z) dz.  s(-z) as 1 - s: where s is near 1 that is off by 2^-24, which the s it is added
    // to outweighs, and where s is small it is exact to rounding.
    const float s = sigmoid(z), f = g * s;
    return {f, __builtin_fmaf(f * (1.0f - s), dz, s)};
}

}  // namespace bsq
