// glu_ops.cuh -- per-element arithmetic of the gated feed-forward kernels (glu.cu), on
// packed float32 pairs (norm_ops.cuh: half the instructions of scalar operations).
//
//     a  = act(g) u                       forward, g and u in FP32
//     dg = dA u act'(g), du = dA act(g)   backward, g and u the stored BF16 values
//
// SiLU g sigma(g); GELU in the tanh form, g (1 + tanh z) / 2 = g sigma(2 z) with
// 2 z = 2 sqrt(2 / pi) (g + 0.044715 g^3), so both take one exponential (base 2: the factor
// log2(e) goes into z's constants) and one reciprocal.  Their derivative is sigma + f (1 -
// sigma) z'(g) with f = g sigma, and z' = 1 for SiLU.  The approximate exponential and
// reciprocal (2 ulp and 1 ulp) are far below the rounding of the result to BF16.
#pragma once

#include "common.cuh"
#include "norm_ops.cuh"

namespace fp8q {

namespace {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGelu2C = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kGelu2CB = 0.07135481282779408f;  // 2 sqrt(2 / pi) 0.044715

__device__ __forceinline__ f32x2 twice(float v) { return pair_of(v, v); }

// 1 / (1 + 2^e); 0 where it is below float32's normal range (e above 126).
__device__ __forceinline__ f32x2 logistic2(f32x2 e) {
    const float2 f = split(e);
    float a, b;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(f.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(f.y));
    const float2 d = split(add2(pair_of(a, b), twice(1.0f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(d.y));
    return pair_of(a, b);
}

__device__ __forceinline__ f32x2 positive2(f32x2 g) {  // max(g, 0), 0 for a NaN
    const float2 f = split(g);
    return pair_of(f.x > 0.0f ? f.x : 0.0f, f.y > 0.0f ? f.y : 0.0f);
}

template <int ACT>
__device__ __forceinline__ f32x2 sigma2(f32x2 g) {
    if constexpr (ACT == FP8Q_ACT_SILU) return logistic2(mul2(g, twice(-kLog2E)));
    return logistic2(mul2(g, fma2(mul2(g, g), twice(-kLog2E * kGelu2CB), twice(-kLog2E * kGelu2C))));
}

template <int ACT>
__device__ __forceinline__ f32x2 glu_act(f32x2 g) {
    if constexpr (ACT == FP8Q_ACT_IDENTITY) return g;
    if constexpr (ACT == FP8Q_ACT_RELU) return positive2(g);
    if constexpr (ACT == FP8Q_ACT_RELU2) {
        const f32x2 p = positive2(g);
        return mul2(p, p);
    }
    return mul2(g, sigma2<ACT>(g));
}

// f = act(g), d = act'(g).
template <int ACT>
__device__ __forceinline__ void glu_act_grad(f32x2 g, f32x2& f, f32x2& d) {
    if constexpr (ACT == FP8Q_ACT_IDENTITY) {
        f = g;
        d = twice(1.0f);
    } else if constexpr (ACT == FP8Q_ACT_RELU) {
        const float2 v = split(g);
        f = positive2(g);
        d = pair_of(v.x > 0.0f ? 1.0f : 0.0f, v.y > 0.0f ? 1.0f : 0.0f);
    } else if constexpr (ACT == FP8Q_ACT_RELU2) {
        const f32x2 p = positive2(g);
        f = mul2(p, p);
        d = add2(p, p);
    } else {
        const f32x2 s = sigma2<ACT>(g);
        f = mul2(g, s);
        f32x2 rest = fma2(s, twice(-1.0f), twice(1.0f));
        if constexpr (ACT == FP8Q_ACT_GELU) {
            // (g^2 held at 2^100: of larger gates, whose squares leave float32, 1 - sigma or f is 0, and 0 times z' has to be)
            const float2 gg = split(mul2(g, g));
            rest = mul2(rest, fma2(pair_of(fminf(gg.x, 0x1p100f), fminf(gg.y, 0x1p100f)), twice(3.0f * kGelu2CB), twice(kGelu2C)));
        }
        d = fma2(f, rest, s);
    }
}

__device__ __forceinline__ uint32_t bf16x2_of(f32x2 v) {
    const float2 f = split(v);
    return cvt_bf16x2(f.x, f.y);
}
__device__ __forceinline__ f32x2 f32x2_of(uint32_t bf16x2) { return pair_of(bf16lo_to_f32(bf16x2), bf16hi_to_f32(bf16x2)); }

}  // namespace

}  // namespace fp8q
