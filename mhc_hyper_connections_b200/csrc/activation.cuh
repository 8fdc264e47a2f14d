// activation.cuh -- the activations of mhc_linear and their slopes, in fp32.
#pragma once

#include "common.cuh"
#include "launch.cuh"

namespace mhc {

constexpr float kSqrtHalf = 0.70710678118654752440f;      // 1 / sqrt(2)
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;    // 1 / sqrt(2 pi)
constexpr float kSqrt8OverPi = 1.59576912160573071176f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// gelu_tanh: (1 + tanh u) / 2 = sigmoid(2 u) with u = sqrt(2/pi) (z + 0.044715 z^3)
__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);     // NaN stays NaN
        case ACT_GELU: return 0.5f * z * (1.0f + erff(z * kSqrtHalf));
        case ACT_GELU_TANH: return z * sigmoid_f32(kSqrt8OverPi * fmaf(kGeluCubic * z * z, z, z));
        case ACT_SILU: return z * sigmoid_f32(z);
        default: return z;
    }
}

__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
        case ACT_RELU: return z > 0.f ? 1.f : (z != z ? z : 0.f);
        case ACT_GELU: return fmaf(z * kInvSqrt2Pi, expf(-0.5f * z * z), 0.5f * (1.0f + erff(z * kSqrtHalf)));
        case ACT_GELU_TANH: {
            const float s = sigmoid_f32(kSqrt8OverPi * fmaf(kGeluCubic * z * z, z, z));
            // past |z| = 9 the slope is 0 or 1 in fp32, and the cubic's derivative may not overflow
            const float q = fminf(z * z, 100.f);
            return fmaf(z * s * (1.0f - s), kSqrt8OverPi * fmaf(3.0f * kGeluCubic, q, 1.0f), s);
        }
        case ACT_SILU: {
            const float s = sigmoid_f32(z);
            return s * fmaf(z, 1.0f - s, 1.0f);
        }
        default: return 1.f;
    }
}

}  // namespace mhc
