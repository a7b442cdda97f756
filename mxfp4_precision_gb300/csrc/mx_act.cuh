// mx_act.cuh -- the activations of a product's epilogue and their derivatives,
// in fp32 (u = 2^-24).
//
// All but ReLU's need one 2^x and one reciprocal (the hardware's, within 2 and
// 1 units in the last place), taken of -|x| so that neither leaves fp32's range:
//   s(t) = 1 / (1 + 2^-t):  e = 2^-|t|, r = 1 / (1 + e);  t >= 0: r, else e r;
//                           s (1 - s) = e r^2, without a difference that cancels
//   silu        x s(x log2 e)
//   gelu_tanh   x s(t), t = 2 sqrt(2/pi) log2 e (x + 0.044715 x^3):
//               (1 + tanh(a)) / 2 = 1 / (1 + exp(-2a))
//   gelu        x Phi(x);  Phi(-|x|) = erfcx(|x| / sqrt 2) / 2 exp(-x^2 / 2)
// with erfcx(w) = exp(w^2) erfc(w) by a polynomial of degree 9 in
// 1 / (1 + 0.3 w), fitted here by reweighted least squares to a relative 3.7e-8 over
// 0 <= w <= 10.5, where exp(-w^2) has left fp32's range.  Phi is within 4 u absolutely;
// relatively within (8 + 3 x^2) u below 0 (the exponent's rounding), so that small
// values of the left tail keep their digits, which 1 + erf(x / sqrt 2) loses.
// Infinities and NaN give what the formulas give (x = -Inf: -Inf * 0 = NaN).
#pragma once

#include <cuda_runtime.h>

namespace mx {
namespace act {

enum : int { kNone = 0, kRelu = 1, kRelu2 = 2, kGelu = 3, kGeluTanh = 4, kSilu = 5 };

__device__ __forceinline__ float exp2_of(float x) {
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(x));
    return e;
}
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// max(x, 0), NaN for NaN.
__device__ __forceinline__ float positive(float x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(0.0f));
    return r;
}

// s(t) and s (1 - s).
struct Sigmoid {
    float s, slope;
};
__device__ __forceinline__ Sigmoid sigmoid(float t) {
    const float e = exp2_of(-fabsf(t)), r = reciprocal(1.0f + e), er = e * r;
    return {t < 0.0f ? er : r, er * r};
}

// Phi(x) and exp(-x^2 / 2).
struct Normal {
    float below, e;
};
__device__ __forceinline__ Normal normal(float x) {
    const float t = reciprocal(fmaf(fabsf(x), 0x1.b27248p-3f, 1.0f));  // 0.3 / sqrt 2
    float p = -0x1.05624cp-4f;
    p = fmaf(p, t, 0x1.e673e6p-3f);
    p = fmaf(p, t, -0x1.f29f92p-3f);
    p = fmaf(p, t, 0x1.06a07ep-2f);
    p = fmaf(p, t, -0x1.093d10p-5f);
    p = fmaf(p, t, 0x1.960778p-4f);
    p = fmaf(p, t, 0x1.3c2144p-4f);
    p = fmaf(p, t, 0x1.5ad880p-4f);
    p = fmaf(p, t, 0x1.5ad9f0p-4f);
    p = fmaf(p, t, -0x1.3ec9bep-18f);
    const float e = exp2_of(x * x * -0x1.715476p-1f);  // log2 e / 2
    const float h = p * e;
    return {x < 0.0f ? h : 1.0f - h, e};
}

constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kTanh = 1.5957691216f;  // 2 sqrt(2/pi)
constexpr float kCubic = 0.044715f;

template <int ACT>
__device__ __forceinline__ float value(float x) {
    if constexpr (ACT == kRelu) return positive(x);
    if constexpr (ACT == kRelu2) {
        const float p = positive(x);
        return p * p;
    }
    if constexpr (ACT == kGelu) return x * normal(x).below;
    if constexpr (ACT == kGeluTanh)
        return x * sigmoid(x * fmaf(x * x, kTanh * kCubic * kLog2e, kTanh * kLog2e)).s;
    if constexpr (ACT == kSilu) return x * sigmoid(x * kLog2e).s;
    return x;
}

template <int ACT>
__device__ __forceinline__ float slope(float x) {
    if constexpr (ACT == kRelu) return x > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == kRelu2) return 2.0f * positive(x);
    if constexpr (ACT == kGelu) {
        const Normal n = normal(x);
        return fmaf(x * n.e, 0.3989422804f, n.below);  // 1 / sqrt(2 pi)
    }
    if constexpr (ACT == kGeluTanh) {
        // Beyond |x| = 10^4 the slope of s is 0; the bound keeps x^2 from making 0 * Inf of it.
        const float x2 = fminf(x * x, 1e8f);
        const Sigmoid q = sigmoid(x * fmaf(x2, kTanh * kCubic * kLog2e, kTanh * kLog2e));
        return fmaf(x * q.slope, fmaf(x2, 3.0f * kTanh * kCubic, kTanh), q.s);
    }
    if constexpr (ACT == kSilu) {
        const Sigmoid q = sigmoid(x * kLog2e);
        return fmaf(x, q.slope, q.s);
    }
    return 1.0f;
}

}  // namespace act
}  // namespace mx
