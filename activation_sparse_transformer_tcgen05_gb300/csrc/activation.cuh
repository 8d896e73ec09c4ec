// activation.cuh — the dense layers' activation functions and their derivatives.
//
//   relu       max(z, 0), derivative [z > 0] (NaN counts as inactive, as in the packed layer)
//   silu       z s(z), s(z) = 1 / (1 + e^-z)
//   gelu       z P(z), P the normal distribution function = (1 + erf(z / sqrt 2)) / 2
//   gelu_tanh  z (1 + tanh i) / 2 = z s(2 i), i = sqrt(2 / pi) (z + 0.044715 z^3)
// All in fp32. The exponential and the quotient are the fast ones: within 4e-7 of
// the value for |z| < 6, where s matters, a hundredth of a bf16 rounding.
#pragma once

#include "common.cuh"

namespace twell {

__device__ __forceinline__ float logistic(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// act(z); da: act'(z).
template <int ACT>
__device__ __forceinline__ float activate(float z, float* da = nullptr)
{
    if constexpr (ACT == TWELL_ACT_RELU) {
        if (da) *da = z > 0.f ? 1.f : 0.f;
        return z > 0.f ? z : 0.f;
    } else if constexpr (ACT == TWELL_ACT_SILU) {
        const float s = logistic(z);
        if (da) *da = s * fmaf(z, 1.f - s, 1.f);
        return z * s;
    } else if constexpr (ACT == TWELL_ACT_GELU) {
        const float p = fmaf(0.5f, erff(z * 0.70710678f), 0.5f);
        if (da) *da = fmaf(z * 0.39894228f, __expf(-0.5f * z * z), p);
        return z * p;
    } else if constexpr (ACT == TWELL_ACT_GELU_TANH) {
        const float k2 = 1.59576912f;  // 2 sqrt(2 / pi)
        const float s = logistic(k2 * fmaf(0.044715f * z * z, z, z));
        if (da) *da = fmaf(z * s * (1.f - s), k2 * fmaf(0.134145f * z, z, 1.f), s);
        return z * s;
    } else {
        if (da) *da = 1.f;
        return z;
    }
}

// f(tag) with the activation as a compile-time value; the choice is uniform over the grid.
template <int V>
struct ActTag {
    static constexpr int value = V;
};
template <class F>
__device__ __forceinline__ void by_activation(int act, F f)
{
    switch (act) {
        case TWELL_ACT_RELU: f(ActTag<TWELL_ACT_RELU>{}); break;
        case TWELL_ACT_SILU: f(ActTag<TWELL_ACT_SILU>{}); break;
        case TWELL_ACT_GELU: f(ActTag<TWELL_ACT_GELU>{}); break;
        case TWELL_ACT_GELU_TANH: f(ActTag<TWELL_ACT_GELU_TANH>{}); break;
        default: f(ActTag<TWELL_ACT_NONE>{}); break;
    }
}

}  // namespace twell
