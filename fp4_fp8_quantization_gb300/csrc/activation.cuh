// The activations of the block product's epilogue and their slopes, fp32.
//
// silu z sigma(z) and the tanh form of gelu, 1/2 z (1 + tanh(w)) = z sigma(2 w), are
// both z sigma(u) with u = z (c1 + c3 z^2).  gelu z Phi(z) takes the normal
// distribution from Abramowitz and Stegun's formula 7.1.26,
//   erfc(x) = (a1 t + .. + a5 t^5) exp(-x^2),  t = 1 / (1 + 0.3275911 x),  x >= 0,
// within 1.5e-7 of it (half of that of Phi).  sigma is within 2^-22, relative to
// itself and to 1 - sigma within 2 + 1.2 |u| ulp of 2^-23 more.
#pragma once

#include "common.cuh"

namespace moeq {

// z sigma(u): the coefficients of u
__device__ __forceinline__ float sigma_c1(int act) {
    return act == MOEQ_ACT_SILU ? 1.0f : 1.5957691216f;  // 2 sqrt(2 / pi)
}
__device__ __forceinline__ float sigma_c3(int act) {
    return act == MOEQ_ACT_SILU ? 0.0f : 0.0713548163f;  // that times 0.044715
}

// z^2, bounded so that it is not infinite times c3 = 0
__device__ __forceinline__ float square(float z) { return fminf(__fmul_rn(z, z), 1e30f); }

// sigma(u) and 1 - sigma(u)
__device__ __forceinline__ void sigma_pair(float u, float &p, float &rest) {
    const float e = __expf(-fabsf(u));
    const float r = __fdividef(1.0f, __fadd_rn(1.0f, e)), er = __fmul_rn(e, r);
    p = u >= 0.0f ? r : er;
    rest = u >= 0.0f ? er : r;
}

// Phi(z) and exp(-z^2 / 2)
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    e = __expf(__fmul_rn(__fmul_rn(-0.5f, z), z));
    const float t = __fdividef(1.0f, __fmaf_rn(fabsf(z), 0.2316418882f, 1.0f));  // 0.3275911 / sqrt 2
    float q = __fmaf_rn(1.061405429f, t, -1.453152027f);
    q = __fmaf_rn(q, t, 1.421413741f);
    q = __fmaf_rn(q, t, -0.284496736f);
    q = __fmaf_rn(q, t, 0.254829592f);
    const float tail = __fmul_rn(__fmul_rn(__fmul_rn(0.5f, q), t), e);
    return z >= 0.0f ? __fadd_rn(1.0f, -tail) : tail;
}

__device__ __forceinline__ float act_sigma(float z, float c1, float c3) {
    const float u = __fmul_rn(z, __fmaf_rn(c3, square(z), c1));
    return __fmul_rn(z, __fdividef(1.0f, __fadd_rn(1.0f, __expf(-u))));
}

__device__ __forceinline__ float act_gelu(float z) {
    float e;
    return __fmul_rn(z, normal_cdf(z, e));
}

// NaN stays NaN
__device__ __forceinline__ float act_relu(float z) { return z <= 0.0f ? 0.0f : z; }

// d act / d z
__device__ __forceinline__ float act_slope(float z, int act, float c1, float c3) {
    if (act == MOEQ_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (act == MOEQ_ACT_GELU) {
        float e;
        const float p = normal_cdf(z, e);
        return __fmaf_rn(__fmul_rn(z, 0.3989422804f), e, p);  // 1 / sqrt(2 pi)
    }
    const float zz = square(z);
    float p, rest;
    sigma_pair(__fmul_rn(z, __fmaf_rn(c3, zz, c1)), p, rest);
    const float du = __fmaf_rn(3.0f * c3, zz, c1);
    return __fmul_rn(p, __fmaf_rn(__fmul_rn(z, du), rest, 1.0f));
}

}  // namespace moeq
