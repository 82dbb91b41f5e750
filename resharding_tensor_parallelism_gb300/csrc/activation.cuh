// The activations of rtp_tp_linear and rtp_tp_glu (rtp_act) and their
// derivatives, in float32 on the float32 accumulator.
//   GELU       x Phi(x);  d = Phi(x) + x phi(x).  Phi(-|x|) = e^(-x^2 / 2) R(|x|), where
//              R(a) = e^(a^2 / 2) Phi(-a) is smooth, falls from 1/2 like 1 / (a sqrt(2 pi)),
//              and is a polynomial of degree 7 in t = 1 / (1 + 0.34 a): weighted least
//              squares on Chebyshev nodes in t, reweighted by the error until it was level
//              (Lawson's method), for |x| up to 14.6, where Phi underflows. In float32 it is
//              within 4e-7 of R up to |x| = 4 and 5e-6 beyond, Phi within 2e-7: the tail is
//              relative to itself, not a difference from 1. Its exponential is that of phi, so
//              value and slope together take one exponential and one quotient. With erff and
//              expf the element-wise step of the linear layer's backward (16384 x 4096) was
//              bound by arithmetic: 168 us.
//   GELU_TANH  x s(2z), z = sqrt(2 / pi) (x + 0.044715 x^3), since (1 + tanh z) / 2 = s(2z),
//              s(v) = 1 / (1 + e^-v); this form keeps its relative accuracy where tanh z is near -1
//   SILU       x s(x);  d = s(x) (1 + x (1 - s(x)))
//   RELU       max(x, 0), a NaN passes;  d = 1 for x > 0
// Values that are rounded to bf16, and slopes, take the approximate exponential below.
// Values that stay float32 (FINE) take expf, and GELU one degree more (c = 0.3, within
// 6e-8 of R, 8e-7 with the roundings) and what float32 drops of x^2: relative to
// themselves they are off by at most 2^-21 (SILU), 2^-19 (GELU), 2^-21 (1 + 2 |z|)
// (GELU_TANH, whose argument is rounded too). 4096 x 512 x 4096, float32, against the
// approximate forms: SILU 32.6 -> 35.7 us, GELU_TANH 33.7 -> 37.5, GELU 34.8 -> 43.1;
// with normcdff and the rounded reciprocal 105, 113 and 97 (bf16 outputs: 33.7, 34.9, 36.1).
#pragma once

#include "rtp.h"

namespace rtp {

namespace {

// e^v and 1 / v by the approximate base-2 exponential and reciprocal instructions
// (2^-22 and 1 ulp; subnormal results and operands count as zero): e^v is off by
// 2^-22 + |v| 2^-24 relative (the rounding of v log2 e; GELU's exponent is rounded
// twice more), at most 2^-15, against bf16's 2^-8.
__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float exp_fast(float v) { return exp2_fast(v * 1.44269504088896340736f); }
__device__ __forceinline__ float rcp_fast(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float logistic(float v) { return rcp_fast(1.0f + exp_fast(-v)); }

constexpr float kTanhScale = 1.5957691216057307f;  // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// Phi(x); e receives e^(-x^2 / 2). FINE: the exponent with the part of x^2 that float32
// drops (|x| is held to 20, where Phi has underflowed, so that x^2 stays finite).
template <bool FINE>
__device__ __forceinline__ float normal_cdf(float x, float& e)
{
    float r;
    if constexpr (FINE) {
        const float a = fminf(fabsf(x), 20.0f), sq = a * a, rest = fmaf(a, a, -sq);
        e = expf(-0.5f * sq);
        e = fmaf(e, -0.5f * rest, e);
        const float t = rcp_fast(1.0f + 0.3f * a);
        r = 7.4024868e-06f + t * (1.19483696e-01f + t * (1.21948972e-01f + t * (9.45713255e-02f + t * (1.42799533e-01f +
            t * (-7.68893970e-02f + t * (2.28995354e-01f + t * (-1.69328611e-01f + t * 3.84117550e-02f)))))));
    } else {
        e = exp2_fast(x * (x * (-0.5f * 1.44269504088896340736f)));
        const float t = rcp_fast(1.0f + 0.34f * fabsf(x));
        r = -5.8135998e-05f + t * (1.3688410e-01f + t * (1.2466286e-01f + t * (1.7229286e-01f + t * (-5.8451386e-02f +
            t * (2.9221521e-01f + t * (-2.1582676e-01f + t * 4.8281305e-02f))))));
    }
    const float tail = r * e;
    return x < 0.0f ? tail : 1.0f - tail;
}

// x s(u) for u of x's sign, float32: s(u) = 1 / (1 + e^-u), or, below 0, e^u / (1 + e^u).
// Below -80 e^u counts as nothing beside 1, and is multiplied in as two halves, so
// that no factor is subnormal before the value is.
__device__ __forceinline__ float logistic_times(float x, float u)
{
    const bool low = u < -80.0f;
    const float e = expf(low ? 0.5f * u : -fabsf(u));
    return (u < 0.0f ? x * e : x) * (low ? e : rcp_fast(1.0f + e));
}

template <int ACT, bool FINE = false>
__device__ __forceinline__ float act_value(float x)
{
    if constexpr (FINE) {
        if constexpr (ACT == RTP_ACT_GELU_TANH) return logistic_times(x, kTanhScale * (x + kTanhCubic * x * x * x));
        if constexpr (ACT == RTP_ACT_SILU) return logistic_times(x, x);
    }
    if constexpr (ACT == RTP_ACT_GELU) {
        float e;
        return x * normal_cdf<FINE>(x, e);
    }
    if constexpr (ACT == RTP_ACT_GELU_TANH) return x * logistic(kTanhScale * (x + kTanhCubic * x * x * x));
    if constexpr (ACT == RTP_ACT_SILU) return x * logistic(x);
    if constexpr (ACT == RTP_ACT_RELU) return x > 0.0f || x != x ? x : 0.0f;
    return x;
}

// a = act(x), d = act'(x)
template <int ACT>
__device__ __forceinline__ void act_both(float x, float& a, float& d)
{
    if constexpr (ACT == RTP_ACT_GELU) {
        float e;
        const float cdf = normal_cdf<false>(x, e);
        a = x * cdf;
        d = cdf + 0.39894228040143267794f * x * e;
    } else if constexpr (ACT == RTP_ACT_GELU_TANH) {
        const float s = logistic(kTanhScale * (x + kTanhCubic * x * x * x));
        const float w = s * (1.0f - s);
        a = x * s;
        // w is zero once the sigmoid has saturated, where x^2 may overflow
        d = s + (w != 0.0f ? x * w * kTanhScale * (1.0f + 3.0f * kTanhCubic * x * x) : 0.0f);
    } else if constexpr (ACT == RTP_ACT_SILU) {
        const float s = logistic(x);
        a = x * s;
        d = s * (1.0f + x * (1.0f - s));
    } else if constexpr (ACT == RTP_ACT_RELU) {
        a = x > 0.0f || x != x ? x : 0.0f;
        d = x > 0.0f ? 1.0f : 0.0f;
    } else {
        a = x;
        d = 1.0f;
    }
}

// Calls body(std::integral_constant-like tag<ACT>) for the runtime `act`: the
// branch is uniform and stands outside the loops over a chunk's elements.
template <int ACT>
struct ActTag {
    static constexpr int value = ACT;
};
template <class Body>
__device__ __forceinline__ void with_act(int act, Body&& body)
{
    switch (act) {
    case RTP_ACT_GELU: body(ActTag<RTP_ACT_GELU>()); break;
    case RTP_ACT_GELU_TANH: body(ActTag<RTP_ACT_GELU_TANH>()); break;
    case RTP_ACT_SILU: body(ActTag<RTP_ACT_SILU>()); break;
    case RTP_ACT_RELU: body(ActTag<RTP_ACT_RELU>()); break;
    default: body(ActTag<RTP_ACT_NONE>()); break;
    }
}

}  // namespace

}  // namespace rtp
