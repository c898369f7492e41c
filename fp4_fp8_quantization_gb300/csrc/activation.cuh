// The activations of the block product's epilogue and their slopes, fp32, two values
// at a time.
//
// silu z sigma(z) and the tanh form of gelu, 1/2 z (1 + tanh(w)) = z sigma(2 w), are
// both z sigma(u), u = z or z (c1 + c3 z^2), and with e = exp(-|u|), r = 1 / (1 + e)
//   sigma(u) = r for u >= 0, e r otherwise;  sigma (1 - sigma) = e r^2.
// gelu z Phi(z) takes the normal distribution from Abramowitz and Stegun's formula
// 7.1.26,
//   erfc(x) = (a1 t + .. + a5 t^5) exp(-x^2),  t = 1 / (1 + 0.3275911 x),  x >= 0,
// within 1.5e-7 of it (half of that of Phi).  An exp(-v) is within 2^-22 + v 2^-23
// relative (2^x to 2 ulp, its argument one product), a reciprocal within 2^-23.
#pragma once

#include "common.cuh"

namespace moeq {

// 2^x and 1 / x of two values (results below 2^-126 are 0).
__device__ __forceinline__ F2 exp2_2(F2 x) {
    float a, b;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(f2_lo(x)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(f2_hi(x)));
    return f2(a, b);
}
__device__ __forceinline__ F2 rcp_2(F2 x) {
    float a, b;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(f2_lo(x)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(f2_hi(x)));
    return f2(a, b);
}

__device__ __forceinline__ F2 abs2(F2 x) { return f2(fabsf(f2_lo(x)), fabsf(f2_hi(x))); }

// x >= 0 ? a : b of each
__device__ __forceinline__ F2 by_sign2(F2 x, F2 a, F2 b) {
    return f2(f2_lo(x) >= 0.0f ? f2_lo(a) : f2_lo(b), f2_hi(x) >= 0.0f ? f2_hi(a) : f2_hi(b));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhC1 = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhC3 = 0.07135481627145224f;  // that times 0.044715

// u of z sigma(u)
template <int ACT>
__device__ __forceinline__ F2 sigma_arg(F2 z, F2 zz) {
    if constexpr (ACT == MOEQ_ACT_SILU) return z;
    return mul2(z, fma2(zz, f2s(kTanhC3), f2s(kTanhC1)));
}

// Phi(z), and exp(-z^2 / 2) in e
__device__ __forceinline__ F2 normal_cdf(F2 z, F2 &e) {
    e = exp2_2(mul2(mul2(z, f2s(-0.5f * kLog2e)), z));
    const F2 t = rcp_2(fma2(abs2(z), f2s(0.23164188839f), f2s(1.0f)));  // 0.3275911 / sqrt 2
    // half of the polynomial
    F2 q = fma2(t, f2s(0.5307027145f), f2s(-0.7265760135f));
    q = fma2(q, t, f2s(0.7107068705f));
    q = fma2(q, t, f2s(-0.142248368f));
    q = fma2(q, t, f2s(0.127414796f));
    const F2 tail = mul2(mul2(q, t), e);
    return by_sign2(z, sub2(f2s(1.0f), tail), tail);
}

// A NaN stays one.
__device__ __forceinline__ float relu(float z) { return z <= 0.0f ? 0.0f : z; }
__device__ __forceinline__ float relu_slope(float z) { return z > 0.0f ? 1.0f : relu(z); }

template <int ACT>
__device__ __forceinline__ F2 activate2(F2 z) {
    if constexpr (ACT == MOEQ_ACT_RELU) return f2(relu(f2_lo(z)), relu(f2_hi(z)));
    if constexpr (ACT == MOEQ_ACT_GELU) {
        F2 e;
        return mul2(z, normal_cdf(z, e));
    }
    if constexpr (ACT == MOEQ_ACT_SILU || ACT == MOEQ_ACT_GELU_TANH) {
        const F2 u = sigma_arg<ACT>(z, mul2(z, z));
        return mul2(z, rcp_2(add2(exp2_2(mul2(u, f2s(-kLog2e))), f2s(1.0f))));
    }
    return z;
}

// d act / d z
template <int ACT>
__device__ __forceinline__ F2 slope2(F2 z) {
    if constexpr (ACT == MOEQ_ACT_RELU) return f2(relu_slope(f2_lo(z)), relu_slope(f2_hi(z)));
    if constexpr (ACT == MOEQ_ACT_GELU) {
        F2 e;
        const F2 p = normal_cdf(z, e);
        return fma2(mul2(z, f2s(0.3989422804f)), e, p);  // 1 / sqrt(2 pi)
    }
    if constexpr (ACT == MOEQ_ACT_SILU || ACT == MOEQ_ACT_GELU_TANH) {
        const F2 zz = mul2(z, z), u = sigma_arg<ACT>(z, zz);
        const F2 e = exp2_2(mul2(abs2(u), f2s(-kLog2e)));
        const F2 r = rcp_2(add2(e, f2s(1.0f))), er = mul2(e, r);
        const F2 d = mul2(er, r), p = by_sign2(u, r, er);
        if constexpr (ACT == MOEQ_ACT_SILU) return fma2(z, d, p);
        // d is 0 from |u| = 88 on; du / dz has to stay finite there (z z is infinite from 2e19
        // on, z du / dz from 1e13), so that the product is 0 too.  NaN for an infinite or NaN z.
        const F2 most = f2(fminf(f2_lo(zz), 1e30f), fminf(f2_hi(zz), 1e30f));
        return fma2(mul2(d, z), fma2(most, f2s(3.0f * kTanhC3), f2s(kTanhC1)), p);
    }
    return f2s(1.0f);
}

}  // namespace moeq
