// What the router's kernels share: logits of the three types as fp32, their
// order as integers, reductions over groups of lanes, a lane's part of a row.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moeq {

constexpr uint32_t kNegInfKey = 0x007FFFFFu;  // order_key(-inf)
constexpr float kInf = __builtin_huge_valf();

template <int DT>
__device__ __forceinline__ float logit_of(uint32_t b) {
    if constexpr (DT == MOEQ_FP32) return __uint_as_float(b);
    if constexpr (DT == MOEQ_BF16) return bf16_bits_to_f32(b);
    return __half2float(__ushort_as_half((unsigned short)b));
}

template <int DT>
__device__ __forceinline__ uint32_t bits_of(float v) {
    if constexpr (DT == MOEQ_FP32) return __float_as_uint(v);
    if constexpr (DT == MOEQ_BF16) return f32_to_bf16_bits(v);
    return __half_as_ushort(__float2half_rn(v));
}

template <int DT>
constexpr int kSize = DT == MOEQ_FP32 ? 4 : 2;

template <int DT>
__device__ __forceinline__ float load_logit(const uint8_t *row, int j) {
    if constexpr (DT == MOEQ_FP32) return __ldg(reinterpret_cast<const float *>(row) + j);
    return logit_of<DT>(__ldg(reinterpret_cast<const uint16_t *>(row) + j));
}

template <int DT>
__device__ __forceinline__ void store_logit(uint8_t *row, int j, float v) {
    if constexpr (DT == MOEQ_FP32)
        reinterpret_cast<float *>(row)[j] = v;
    else
        reinterpret_cast<uint16_t *>(row)[j] = (uint16_t)bits_of<DT>(v);
}

// An integer that orders as the float, no NaN, does (-0 = +0).
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// exp(x - m) for x <= m: with d the difference rounded to fp32, within
// 2 + 1.2 |d| ulp of exp(d), to which the rounding adds |d| 2^-24 of the value.
// NaN for a NaN or for infinity minus infinity.
__device__ __forceinline__ float exp_diff(float x, float m) { return __expf(__fadd_rn(x, -m)); }

// Maximum over groups of LANES consecutive lanes, the same in each of them.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (LANES == 32) return __reduce_max_sync(0xFFFFFFFFu, v);
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Sum over groups of LANES consecutive lanes, the same in each of them.
template <int LANES = 32>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Whether every row starts where vectors of a lane's logits (16 bytes at
// most) can be read and written.
template <int DT, int NV>
__device__ __forceinline__ bool rows_aligned(int64_t stride) {
    constexpr int kBytes = NV * kSize<DT> < 16 ? NV * kSize<DT> : 16;
    return stride % kBytes == 0;
}

// The lane's logits; -inf past the row's end.
template <int DT, int NV>
__device__ __forceinline__ void load_row(const uint8_t *row, int E, int j0, bool vec,
                                         float (&x)[NV]) {
    constexpr int kBytes = NV * kSize<DT>;
    if (vec && j0 + NV <= E) {
        const uint8_t *a = row + (int64_t)j0 * kSize<DT>;
        uint32_t w[kBytes < 4 ? 1 : kBytes / 4];
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(a) + i);
                w[4 * i] = u.x;
                w[4 * i + 1] = u.y;
                w[4 * i + 2] = u.z;
                w[4 * i + 3] = u.w;
            }
        } else if constexpr (kBytes == 8) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(a));
            w[0] = u.x;
            w[1] = u.y;
        } else if constexpr (kBytes == 4) {
            w[0] = __ldg(reinterpret_cast<const uint32_t *>(a));
        } else {
            w[0] = __ldg(reinterpret_cast<const uint16_t *>(a));
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            x[i] = logit_of<DT>(DT == MOEQ_FP32 ? w[i * kSize<DT> / 4]
                                                : (w[i / 2] >> (16 * (i & 1))) & 0xFFFFu);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = j0 + i < E ? load_logit<DT>(row, j0 + i) : -kInf;
    }
}

}  // namespace moeq
