// activation.cuh — the dense layers' activation functions and their derivatives.
//
//   relu       max(z, 0), derivative [z > 0] (NaN counts as inactive, as in the packed layer)
//   silu       z s(z), s(z) = 1 / (1 + e^-z)
//   gelu       z P(z), P the normal distribution function; derivative P(z) + z e^(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z (1 + tanh i) / 2 = z s(2 i), i = sqrt(2 / pi) (z + 0.044715 z^3)
// All in fp32. The exponential and the quotient are the fast ones: within 4e-7 of
// the value for |z| < 6, where s matters, a hundredth of a bf16 rounding. P's tail is a
// polynomial t (c1 + ... + c6 t^5) in t = 1 / (1 + 0.29 |z|) times the e^(-z^2 / 2) that
// the derivative needs anyway. The coefficients are a fit (iteratively reweighted least
// squares) to the tail times e^(z^2 / 2) on |z| < 14, under both bounds at once: within
// 6e-8, and within 1.2e-4 of the tail itself, a thirtieth of a bf16 rounding. (The five
// terms of Abramowitz and Stegun 7.1.26 are within 8e-8, but 0.4 % off the tail at z = -6
// and 2 % at -10; five terms under both bounds, 5e-7. With erff, and eight warps, the
// epilogue of the backward's first product was longer than the product itself: 777 x 1000 x
// 2696 37 us, now 24.)
#pragma once

#include "common.cuh"

namespace twell {

// (of 1 to infinity)
__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 exp2_pair(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float2 reciprocal_pair(float2 x) { return make_float2(reciprocal(x.x), reciprocal(x.y)); }

// act(z) of two values, for the instructions that work on two at once (half the instructions of the epilogues, and of
// the pass over dy and the pre-activations); da: act'(z).
template <int ACT>
__device__ __forceinline__ float2 activate(float2 z, float2* da = nullptr)
{
    if constexpr (ACT == TWELL_ACT_RELU) {
        if (da) *da = make_float2(z.x > 0.f ? 1.f : 0.f, z.y > 0.f ? 1.f : 0.f);
        return make_float2(z.x > 0.f ? z.x : 0.f, z.y > 0.f ? z.y : 0.f);
    } else if constexpr (ACT == TWELL_ACT_SILU) {
        const float2 s = reciprocal_pair(__fadd2_rn(exp2_pair(__fmul2_rn(z, pair(-1.44269504f))), pair(1.f)));
        if (da) *da = __fmul2_rn(s, __ffma2_rn(z, __ffma2_rn(s, pair(-1.f), pair(1.f)), pair(1.f)));
        return __fmul2_rn(z, s);
    } else if constexpr (ACT == TWELL_ACT_GELU) {
        const float2 e = exp2_pair(__fmul2_rn(__fmul2_rn(z, z), pair(-0.72134752f)));  // e^(-z^2 / 2)
        const float2 t = reciprocal_pair(__ffma2_rn(make_float2(fabsf(z.x), fabsf(z.y)), pair(0.29f), pair(1.f)));
        float2 q = __ffma2_rn(t, pair(-0.0891031250f), pair(0.285923600f));
        q = __ffma2_rn(t, q, pair(-0.0946542323f));
        q = __ffma2_rn(t, q, pair(0.180511311f));
        q = __ffma2_rn(t, q, pair(0.100418434f));
        q = __fmul2_rn(__fmul2_rn(__ffma2_rn(t, q, pair(0.116904020f)), t), e);
        const float2 o = __ffma2_rn(q, pair(-1.f), pair(1.f));
        const float2 p = make_float2(z.x < 0.f ? q.x : o.x, z.y < 0.f ? q.y : o.y);
        if (da) *da = __ffma2_rn(__fmul2_rn(z, pair(0.39894228f)), e, p);
        return __fmul2_rn(z, p);
    } else if constexpr (ACT == TWELL_ACT_GELU_TANH) {
        const float k = 1.59576912f;  // 2 sqrt(2 / pi)
        // (below the squares that pass fp32's range: times the 0 of s (1 - s) those would be NaN in the derivative)
        const float2 sq = __fmul2_rn(z, z), z2 = make_float2(fminf(sq.x, 1e30f), fminf(sq.y, 1e30f));
        const float2 i = __fmul2_rn(__ffma2_rn(z2, pair(-1.44269504f * k * 0.044715f), pair(-1.44269504f * k)), z);
        const float2 s = reciprocal_pair(__fadd2_rn(exp2_pair(i), pair(1.f))), zs = __fmul2_rn(z, s);
        if (da)
            *da = __ffma2_rn(__fmul2_rn(zs, __ffma2_rn(s, pair(-1.f), pair(1.f))),
                             __ffma2_rn(z2, pair(k * 0.134145f), pair(k)), s);
        return zs;
    } else {
        if (da) *da = pair(1.f);
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
