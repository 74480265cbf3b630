// activation.cuh -- the activations of the fused linear layer and of the
// expert layer, and their derivatives, in fp32.
//
//   relu       max(0, z); a NaN stays a NaN
//   gelu       z Phi(z), Phi the normal distribution function
//   gelu_tanh  z / (1 + exp(-2 u)), u = sqrt(2 / pi) (z + 0.044715 z^3)
//              (the tanh form: (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)))
//   silu       z / (1 + exp(-z))
// At z = -inf the last three take their limit 0 (the formulas give
// -inf * 0), and their derivatives the limits 0 and 1 at -inf and +inf.
#pragma once
#include <cstdint>

namespace gbr {

enum Act : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };
constexpr int kActs = 5;

constexpr float kSqrtHalf = 0.70710678118654752440f;      // 1 / sqrt(2)
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;    // 1 / sqrt(2 pi)
constexpr float kSqrt2OverPi = 0.79788456080286535588f;   // sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;
// Beyond |z| = 40 Phi(z), its density and the logistic function are 0 or 1 in
// fp32 to the last bit of the product with z.
constexpr float kActTail = 40.f;

__device__ __forceinline__ float logistic(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// Phi(z), given e = exp(-z^2 / 2): formula 7.1.26 of Abramowitz and Stegun,
// "Handbook of Mathematical Functions" (1964), erfc(x) ~ t (a1 + t (a2 + ...))
// exp(-x^2) with t = 1 / (1 + 0.3275911 x), off by at most 1.5e-7, taken at
// x = |z| / sqrt(2).  One exponential serves Phi and the density, and nothing
// cancels for z < 0.
__device__ __forceinline__ float normal_cdf(float z, float e) {
    const float t = __fdividef(1.f, fmaf(0.3275911f * kSqrtHalf, fabsf(z), 1.f));
    float p = fmaf(t, 1.061405429f, -1.453152027f);
    p = fmaf(t, p, 1.421413741f);
    p = fmaf(t, p, -0.284496736f);
    p = fmaf(t, p, 0.254829592f);
    const float q = 0.5f * t * p * e;
    return z > 0.f ? 1.f - q : q;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == kActRelu) return z <= 0.f ? 0.f : z;
    if (ACT == kActGelu) return z < -kActTail ? 0.f : z * normal_cdf(z, __expf(-0.5f * z * z));
    if (ACT == kActGeluTanh) {
        const float u = kSqrt2OverPi * (z + kGeluCubic * z * z * z);
        return z < -kActTail ? 0.f : z * logistic(2.f * u);
    }
    if (ACT == kActSilu) return z < -kActTail ? 0.f : z * logistic(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if (ACT == kActRelu) return z > 0.f ? 1.f : 0.f;
    if (ACT == kActNone) return 1.f;
    float d;
    if (ACT == kActGelu) {
        const float e = __expf(-0.5f * z * z);
        d = fmaf(z * kInvSqrt2Pi, e, normal_cdf(z, e));
    } else if (ACT == kActGeluTanh) {
        const float s = logistic(2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
        d = s + 2.f * z * s * (1.f - s) * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * z * z);
    } else {
        const float q = logistic(z);
        d = q + z * q * (1.f - q);
    }
    d = z > kActTail ? 1.f : d;
    return z < -kActTail ? 0.f : d;
}

// The same with the activation as a run-time value (uniform over the launch).
__device__ __forceinline__ float act_value(int act, float z) {
    switch (act) {
        case kActRelu: return act_value<kActRelu>(z);
        case kActGelu: return act_value<kActGelu>(z);
        case kActGeluTanh: return act_value<kActGeluTanh>(z);
        case kActSilu: return act_value<kActSilu>(z);
        default: return z;
    }
}

}  // namespace gbr
