// activation.cuh -- the activations of mhc_linear and their slopes, in fp32.
//
// FAST = false, for fp32 storage, evaluates them with the accurate library functions.  FAST = true,
// for bf16 storage, stays within 2^-15.9 of every value that is a normal number (of 1 + the value, for
// slopes, 2^-19; measured at 5e6 points of [-100, 100]), a 240th of the rounding that follows, at about a third of the instructions: the hardware's exponential and
// division, and the normal distribution function from
//     erfc(x) = exp(-x^2) t P(t),  t = 1 / (1 + 0.38 x),  x >= 0,
// with P of degree 6 fitted to exp(x^2) erfc(x) on [0, 10] for the smallest relative error (1.03e-6;
// past 10 both sides are below 1e-44).  Unlike erff this has no branch, and the exponential is the
// one the slope's density needs.  Measured on the forward product of T = 16384, 4096 -> 16384 with
// GELU: see linear_tc.cu.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "launch.cuh"

namespace mhc {

constexpr float kSqrtHalf = 0.70710678118654752440f;      // 1 / sqrt(2)
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;    // 1 / sqrt(2 pi)
constexpr float kSqrt8OverPi = 1.59576912160573071176f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

constexpr float kLog2e = 1.44269504088896340736f;

// the hardware's 2^x and 1 / x
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool FAST>
__device__ __forceinline__ float act_sigmoid(float z) {
    if constexpr (FAST) return rcp_approx(1.0f + ex2_approx(-kLog2e * z));
    return sigmoid_f32(z);
}

// z sigmoid(u), for an activation's value: sigmoid(u) may be below the normal numbers, or exp(-u) above them,
// where the product is not (SiLU of -88 is -5.3e-37, and came out as 0 from z sigmoid(z)).  FAST divides
// 2^-8 z by 2^-8 (1 + exp(-u)); the other form takes exp(-u) as a square.
template <bool FAST>
__device__ __forceinline__ float times_sigmoid(float z, float u) {
    if constexpr (FAST) return (0x1p-8f * z) * rcp_approx(0x1p-8f + ex2_approx(fmaf(-kLog2e, u, -8.0f)));
    const float h = expf(-0.5f * fabsf(u)), r = 1.0f / fmaf(h, h, 1.0f);
    return u < 0.f ? (z * h) * (h * r) : z * r;        // u NaN: r is NaN
}

// Phi(z), and exp(-z^2 / 2)
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    if constexpr (FAST) {
        e = ex2_approx((-0.5f * kLog2e * z) * z);
        const float t = rcp_approx(fmaf(0.38f * kSqrtHalf, fabsf(z), 1.0f));
        float p = 0.5f * -0.12520070f;                     // P / 2
        p = fmaf(p, t, 0.5f * 0.33520198f);
        p = fmaf(p, t, 0.5f * -0.06861920f);
        p = fmaf(p, t, 0.5f * 0.24680305f);
        p = fmaf(p, t, 0.5f * 0.18103781f);
        p = fmaf(p, t, 0.5f * 0.21648033f);
        p = fmaf(p, t, 0.5f * 0.21429573f);
        const float tail = t * p * e;                      // Phi(-|z|)
        return z > 0.f ? 1.0f - tail : tail;
    } else {
        e = expf(-0.5f * z * z);
        // the small side from erfc, so that it keeps its relative accuracy (1 + erf cancels there: off by a
        // fifth at z = -5)
        const float tail = 0.5f * erfcf(fabsf(z) * kSqrtHalf);
        return z > 0.f ? 1.0f - tail : (z != z ? z : tail);
    }
}

// gelu_tanh: (1 + tanh u) / 2 = sigmoid(2 u) with u = sqrt(2/pi) (z + 0.044715 z^3)
template <int ACT, bool FAST>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);     // NaN stays NaN
    if constexpr (ACT == ACT_GELU) {
        float e;
        return z * normal_cdf<FAST>(z, e);
    }
    if constexpr (ACT == ACT_GELU_TANH) return times_sigmoid<FAST>(z, kSqrt8OverPi * fmaf(kGeluCubic * z * z, z, z));
    if constexpr (ACT == ACT_SILU) return times_sigmoid<FAST>(z, z);
    return z;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
    if constexpr (ACT == ACT_GELU) {
        float e;
        const float cdf = normal_cdf<FAST>(z, e);
        return fmaf(z * kInvSqrt2Pi, e, cdf);
    }
    if constexpr (ACT == ACT_GELU_TANH) {
        const float s = act_sigmoid<FAST>(kSqrt8OverPi * fmaf(kGeluCubic * z * z, z, z));
        // past |z| = 10 the slope is 0 or 1 in fp32, and the cubic's derivative may not overflow
        const float q = fminf(z * z, 100.f);
        return fmaf(z * s * (1.0f - s), kSqrt8OverPi * fmaf(3.0f * kGeluCubic, q, 1.0f), s);
    }
    if constexpr (ACT == ACT_SILU) {
        const float s = act_sigmoid<FAST>(z);
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    return 1.f;
}

// f(integral_constant<int, act>): the choice of the activation, outside the loops over elements
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case ACT_RELU: f(std::integral_constant<int, ACT_RELU>{}); break;
        case ACT_GELU: f(std::integral_constant<int, ACT_GELU>{}); break;
        case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>{}); break;
        case ACT_SILU: f(std::integral_constant<int, ACT_SILU>{}); break;
        default: f(std::integral_constant<int, ACT_NONE>{}); break;
    }
}

}  // namespace mhc
