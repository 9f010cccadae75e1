// glu_ops.cuh -- per-element arithmetic of the gated feed-forward kernels (glu.cu).
//
//     a  = act(g) u                       forward, g and u in FP32
//     dg = dA u act'(g), du = dA act(g)   backward, g and u the stored BF16 values
//
// SiLU g sigma(g); GELU in the tanh form, g (1 + tanh z) / 2 = g sigma(2 z) with
// 2 z = 2 sqrt(2 / pi) (g + 0.044715 g^3), so both take one exponential and one
// reciprocal.  Their derivative is sigma + g sigma (1 - sigma) z'(g) with z' = 1 for
// SiLU.  The fast exponential and division (about 2 ulp each) are far below the
// rounding of the result to BF16.
#pragma once

#include "common.cuh"

namespace fp8q {

namespace {

constexpr float kGelu2C = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kGelu2CB = 0.07135481282779408f;  // 2 sqrt(2 / pi) 0.044715

__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float glu_act(float g) {
    if constexpr (ACT == FP8Q_ACT_IDENTITY) return g;
    const float p = g > 0.0f ? g : 0.0f;
    if constexpr (ACT == FP8Q_ACT_RELU) return p;
    if constexpr (ACT == FP8Q_ACT_RELU2) return p * p;
    if constexpr (ACT == FP8Q_ACT_SILU) return g * logistic(g);
    return g * logistic(g * (kGelu2C + kGelu2CB * g * g));
}

// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ float2 glu_act_grad(float g) {
    if constexpr (ACT == FP8Q_ACT_IDENTITY) return make_float2(g, 1.0f);
    const float p = g > 0.0f ? g : 0.0f;
    if constexpr (ACT == FP8Q_ACT_RELU) return make_float2(p, g > 0.0f ? 1.0f : 0.0f);
    if constexpr (ACT == FP8Q_ACT_RELU2) return make_float2(p * p, 2.0f * p);
    const float g2 = g * g;
    const float z = ACT == FP8Q_ACT_SILU ? g : g * (kGelu2C + kGelu2CB * g2);
    const float dz = ACT == FP8Q_ACT_SILU ? 1.0f : kGelu2C + 3.0f * kGelu2CB * g2;
    const float s = logistic(z), f = g * s;
    // where the exponential runs over (z below -88) s is 0 and f a zero; z' may be large, not infinite
    return make_float2(f, s + f * (1.0f - s) * dz);
}

}  // namespace

}  // namespace fp8q
