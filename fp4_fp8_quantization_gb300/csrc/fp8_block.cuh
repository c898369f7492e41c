// The steps of the FP8 quantizers with one scale for many elements: s = max(amax
// / 448, 2^-126), q = E4M3(x * (1 / s)), each one fp32 operation.
#pragma once

#include "common.cuh"

namespace moeq {

__device__ __forceinline__ float block_scale(float amax) {
    return fmaxf(__fdiv_rn(amax, 448.0f), __uint_as_float(0x00800000u));
}

// fmaxf drops a NaN operand, so a NaN never becomes the amax.
__device__ __forceinline__ float amax8(const float (&x)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    return m;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float r) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], r);
    return make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16),
                      e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

}  // namespace moeq
