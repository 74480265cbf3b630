// activation.cuh -- the activations of the fused linear layer and of the
// expert layer, and their derivatives, in fp32.
//
//   relu       max(0, z); a NaN stays a NaN
//   gelu       z Phi(z), Phi the normal distribution function
//   gelu_tanh  z / (1 + exp(-2 u)), u = sqrt(2 / pi) (z + 0.044715 z^3)
//              (the tanh form: (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)))
//   silu       z / (1 + exp(-z))
// At z = -inf the last three take their limit 0, and their derivatives the
// limits 0 and 1 at -inf and +inf.
#pragma once
#include <cstdint>

namespace gbr {

enum Act : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };
constexpr int kActs = 5;

constexpr float kSqrtHalf = 0.70710678118654752440f;      // 1 / sqrt(2)
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;    // 1 / sqrt(2 pi)
constexpr float kSqrt2OverPi = 0.79788456080286535588f;   // sqrt(2 / pi)
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kGeluCubic = 0.044715f;
// At |z| = 100 exp(z) and exp(-z^2 / 2) have left fp32, so that Phi, its
// density and the logistic function are exactly 0 or 1: clamping z there gives
// the limits at +-inf, where the formulas would multiply inf by 0.
constexpr float kActTail = 100.f;

// Two fp32 values in a 64-bit register: one instruction multiplies or adds
// both.  4096 x 14336 derivatives of GELU with their column sums: 85 us with
// one at a time, 58 with two (ReLU, next to no arithmetic: 42).
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split2(F2 x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ F2 exp2_2(F2 x) {
    float a, b;
    split2(x, a, b);
    return f2(exp2_approx(a), exp2_approx(b));
}
__device__ __forceinline__ F2 rcp2(F2 x) {
    float a, b;
    split2(x, a, b);
    return f2(rcp_approx(a), rcp_approx(b));
}
// Larger and smaller of two, a NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// 1 / (1 + exp(-x)).
__device__ __forceinline__ F2 logistic2(F2 x) {
    return rcp2(add2(f2(1.f), exp2_2(mul2(x, f2(-kLog2e)))));
}

// Phi(z), given e = exp(-z^2 / 2): formula 7.1.26 of Abramowitz and Stegun,
// "Handbook of Mathematical Functions" (1964), erfc(x) ~ t (a1 + t (a2 + ...))
// exp(-x^2) with t = 1 / (1 + 0.3275911 x), off by at most 1.5e-7 (absolute), taken at
// x = |z| / sqrt(2) and halved.  One exponential serves Phi and the density,
// and nothing cancels for z < 0.
__device__ __forceinline__ F2 normal_cdf2(F2 z, F2 e) {
    float z0, z1, q0, q1;
    split2(z, z0, z1);
    const F2 t = rcp2(fma2(f2(fabsf(z0), fabsf(z1)), f2(0.3275911f * kSqrtHalf), f2(1.f)));
    F2 p = fma2(t, f2(0.5f * 1.061405429f), f2(0.5f * -1.453152027f));
    p = fma2(t, p, f2(0.5f * 1.421413741f));
    p = fma2(t, p, f2(0.5f * -0.284496736f));
    p = fma2(t, p, f2(0.5f * 0.254829592f));
    const F2 q = mul2(mul2(t, p), e);
    split2(q, q0, q1);
    return f2(z0 > 0.f ? 1.f - q0 : q0, z1 > 0.f ? 1.f - q1 : q1);
}

// Two pre-activations to their activations, in place.
template <int ACT>
__device__ __forceinline__ void act_value2(float& a, float& b) {
    if (ACT == kActRelu) {
        a = a <= 0.f ? 0.f : a;
        b = b <= 0.f ? 0.f : b;
    }
    if (ACT == kActRelu || ACT == kActNone) return;
    const F2 z = f2(max_nan(a, -kActTail), max_nan(b, -kActTail));
    F2 s;
    if (ACT == kActGelu) {
        s = normal_cdf2(z, exp2_2(mul2(mul2(z, z), f2(-0.5f * kLog2e))));
    } else if (ACT == kActGeluTanh) {
        // 2 u = 2 sqrt(2 / pi) z (1 + 0.044715 z^2)
        s = logistic2(mul2(z, fma2(mul2(z, z), f2(2.f * kSqrt2OverPi * kGeluCubic), f2(2.f * kSqrt2OverPi))));
    } else {
        s = logistic2(z);
    }
    split2(mul2(z, s), a, b);
}

// Two gradients times the activation's derivative at their pre-activations.
template <int ACT>
__device__ __forceinline__ void act_slope2(float& a, float& b, float za, float zb) {
    if (ACT == kActRelu) {
        a = za > 0.f ? a : 0.f * a;
        b = zb > 0.f ? b : 0.f * b;
    }
    if (ACT == kActRelu || ACT == kActNone) return;
    const F2 z = f2(min_nan(max_nan(za, -kActTail), kActTail), min_nan(max_nan(zb, -kActTail), kActTail));
    F2 d;
    if (ACT == kActGelu) {
        const F2 e = exp2_2(mul2(mul2(z, z), f2(-0.5f * kLog2e)));
        d = fma2(mul2(z, f2(kInvSqrt2Pi)), e, normal_cdf2(z, e));
    } else if (ACT == kActGeluTanh) {
        const F2 zz = mul2(z, z);
        const F2 s = logistic2(mul2(z, fma2(zz, f2(2.f * kSqrt2OverPi * kGeluCubic), f2(2.f * kSqrt2OverPi))));
        // s + z s (1 - s) 2 u', u' = sqrt(2 / pi) (1 + 3 * 0.044715 z^2)
        const F2 u = fma2(zz, f2(6.f * kSqrt2OverPi * kGeluCubic), f2(2.f * kSqrt2OverPi));
        d = fma2(mul2(mul2(z, u), s), fma2(s, f2(-1.f), f2(1.f)), s);
    } else {
        const F2 s = logistic2(z);
        d = fma2(mul2(z, s), fma2(s, f2(-1.f), f2(1.f)), s);
    }
    split2(mul2(f2(a, b), d), a, b);
}

}  // namespace gbr
