// mx_act.cuh -- the activations of a product's epilogue and their derivatives,
// in fp32 (u = 2^-24), two columns at a time (the f32x2 instructions round each
// half like the scalar ones, at half the issue slots).
//
// silu, gelu_tanh and gelu are x less the part that a factor 1 - h takes away, with h
// of |x| so that nothing leaves fp32's range or cancels:
//   act(x) = x [x > 0] - |x| h(|x|)
//   silu        h = e r,  e = 2^(-|x| log2 e),  r = 1 / (1 + e)     (1 - h = r)
//   gelu_tanh   the same with e = 2^-t, t = 2 sqrt(2/pi) log2 e (|x| + 0.044715 |x|^3):
//               (1 + tanh(a)) / 2 = 1 / (1 + exp(-2a))
//   gelu        h = Phi(-|x|) = erfcx(|x| / sqrt 2) / 2 * e,  e = exp(-x^2 / 2)
// one 2^x and one reciprocal each (the hardware's, within 2 and 1 units in the last
// place).  2^y is the square of 2^(y/2), which keeps values below fp32's normal range.
// erfcx(w) = exp(w^2) erfc(w) is a polynomial of degree 9 in 1 / (1 + 0.3 w),
// fitted here by reweighted least squares to a relative 3.7e-8 over 0 <= w <= 10.5,
// where exp(-w^2) has left fp32's range.  h is relatively within (12 + 3 x^2) u (the
// exponent's rounding), so small values of the left tail keep their digits, which
// 1 + erf(x / sqrt 2) loses.  |x| is held to 32 inside h, which is below fp32's range from there
// on (silu: to 128).  x = -Inf gives the formulas' -Inf * 0 = NaN.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mx_encode.cuh"

namespace mx {
namespace act {

enum : int { kNone = 0, kRelu = 1, kRelu2 = 2, kGelu = 3, kGeluTanh = 4, kSilu = 5 };

using enc::add2;
using enc::mul2;
using enc::pack2;
using enc::unpack2;
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t same2(float v) { return pack2(v, v); }

__device__ __forceinline__ float exp2_of(float x) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
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
// 1 where x > 0, else 0.
__device__ __forceinline__ float step(float x) {
    float r;
    asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(0.0f));
    return r;
}
// The same, NaN for NaN: max(step(x), min(x, 0)).
__device__ __forceinline__ float step_or_nan(float x) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(0.0f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(step(x)));
    return r;
}
__device__ __forceinline__ uint64_t step2(uint64_t x) {
    float a, b;
    unpack2(x, a, b);
    return pack2(step(a), step(b));
}
// max(-|x|, -most); -most for NaN.
__device__ __forceinline__ uint64_t bounded2(uint64_t x, float most) {
    float a, b;
    unpack2(x, a, b);
    return pack2(fmaxf(-fabsf(a), -most), fmaxf(-fabsf(b), -most));
}
// 2^(2 y).
__device__ __forceinline__ uint64_t exp2_twice2(uint64_t y) {
    float a, b;
    unpack2(y, a, b);
    const uint64_t e = pack2(exp2_of(a), exp2_of(b));
    return mul2(e, e);
}
__device__ __forceinline__ uint64_t reciprocal2(uint64_t x) {
    float a, b;
    unpack2(x, a, b);
    return pack2(reciprocal(a), reciprocal(b));
}

constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kTanh = 1.5957691216f;  // 2 sqrt(2/pi)
constexpr float kCubic = 0.044715f;

// Of n = -|x|: h, and what its derivative needs (logistic forms: r; gelu: exp(-x^2 / 2)).
struct Part {
    uint64_t h, more;
};
template <int ACT>
__device__ __forceinline__ Part part2(uint64_t n) {
    if constexpr (ACT == kGelu) {
        const uint64_t t = reciprocal2(fma2(n, same2(-0x1.b27248p-3f), same2(1.0f)));  // 0.3 / sqrt 2
        uint64_t p = same2(-0x1.05624cp-4f);
        p = fma2(p, t, same2(0x1.e673e6p-3f));
        p = fma2(p, t, same2(-0x1.f29f92p-3f));
        p = fma2(p, t, same2(0x1.06a07ep-2f));
        p = fma2(p, t, same2(-0x1.093d10p-5f));
        p = fma2(p, t, same2(0x1.960778p-4f));
        p = fma2(p, t, same2(0x1.3c2144p-4f));
        p = fma2(p, t, same2(0x1.5ad880p-4f));
        p = fma2(p, t, same2(0x1.5ad9f0p-4f));
        p = fma2(p, t, same2(-0x1.3ec9bep-18f));
        const uint64_t e = exp2_twice2(mul2(mul2(n, n), same2(-0.25f * kLog2e)));
        return {mul2(p, e), e};
    } else {
        uint64_t y;
        if constexpr (ACT == kGeluTanh)
            y = mul2(n, fma2(mul2(n, n), same2(0.5f * kTanh * kCubic * kLog2e), same2(0.5f * kTanh * kLog2e)));
        else
            y = mul2(n, same2(0.5f * kLog2e));
        const uint64_t e = exp2_twice2(y), r = reciprocal2(add2(e, same2(1.0f)));
        return {mul2(e, r), r};
    }
}
template <int ACT>
__device__ __forceinline__ constexpr float most() {
    return ACT == kSilu ? 128.0f : 32.0f;
}

// act(x) of two columns.
template <int ACT>
__device__ __forceinline__ uint64_t value2(uint64_t x) {
    if constexpr (ACT == kRelu || ACT == kRelu2) {
        float a, b;
        unpack2(x, a, b);
        const uint64_t p = pack2(positive(a), positive(b));
        return ACT == kRelu ? p : mul2(p, p);
    } else if constexpr (ACT == kNone) {
        return x;
    } else {
        const uint64_t n = bounded2(x, most<ACT>());
        return fma2(x, step2(x), mul2(n, part2<ACT>(n).h));
    }
}

// act'(x) of two columns: s' = s + x s (1 - s) c for the logistic forms, s = [x > 0] + sign h;
// Phi(x) + x phi(x) for gelu.  h and the second term are even and odd in x.  NaN stays NaN.
template <int ACT>
__device__ __forceinline__ uint64_t slope2(uint64_t x) {
    if constexpr (ACT == kRelu || ACT == kRelu2) {
        float a, b;
        unpack2(x, a, b);
        return ACT == kRelu ? pack2(step_or_nan(a), step_or_nan(b)) : mul2(same2(2.0f), pack2(positive(a), positive(b)));
    }
    if constexpr (ACT == kNone) return same2(1.0f);
    const uint64_t n = bounded2(x, most<ACT>());
    const Part q = part2<ACT>(n);
    uint64_t low;  // the slope at -|x|: h - |x| (-h')
    if constexpr (ACT == kGelu) low = fma2(mul2(n, q.more), same2(0.3989422804f), q.h);  // 1 / sqrt(2 pi)
    else if constexpr (ACT == kSilu) low = fma2(n, mul2(q.h, q.more), q.h);
    else low = fma2(mul2(n, mul2(q.h, q.more)), fma2(mul2(n, n), same2(3.0f * kTanh * kCubic), same2(kTanh)), q.h);
    float u, v, xa, xb;
    unpack2(low, u, v);
    unpack2(x, xa, xb);
    // x > 0: 1 - low; NaN stays NaN.
    u = xa > 0.0f ? 1.0f - u : xa <= 0.0f ? u : xa;
    v = xb > 0.0f ? 1.0f - v : xb <= 0.0f ? v : xb;
    return pack2(u, v);
}

}  // namespace act
}  // namespace mx
