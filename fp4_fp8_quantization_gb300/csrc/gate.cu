// The router: top-k choice of each token's expert logits and the softmax
// weights of the chosen, and its gradient.  With x the logits of a token,
// m = max x, i_1 .. i_k its choices (largest logits first, ties to the lowest
// index), s the scale:
//
//   p_j = exp(x_j - m) / sum_l exp(x_l - m)
//   w_r = s p_{i_r}                          or, normalised,
//   w_r = s exp(x_{i_r} - m) / sum_c exp(x_{i_c} - m)
//   d_x = p (g - <p, g>),  g_j = sum_{r: i_r = j} s d_w_r       (plain)
//   d_x_{i_r} = s q_r (d_w_r - <q, d_w>), 0 elsewhere, q = w / s  (normalised)
//
// One warp per token with the whole row of logits in registers (E <= 1024),
// one pass over memory each way.  Selection compares order-preserving integer
// images of the logits: each round is one warp maximum of those and one
// minimum of the indices that hold it.  exp is the library's own (common.cuh);
// sums are fp32 in a fixed order.
#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.h"

namespace moeq {

namespace {

constexpr uint32_t kNegInfKey = 0x007FFFFFu;  // order_key(-inf)
constexpr int kGateWarps = 4;

template <int DT>
__device__ __forceinline__ float load_logit(const void *row, int j) {
    if constexpr (DT == MOEQ_FP32) return __ldg(static_cast<const float *>(row) + j);
    const uint16_t b = __ldg(static_cast<const uint16_t *>(row) + j);
    if constexpr (DT == MOEQ_BF16) return bf16_bits_to_f32(b);
    return __half2float(__ushort_as_half(b));
}

template <int DT>
__device__ __forceinline__ void store_logit(void *row, int j, float v) {
    if constexpr (DT == MOEQ_FP32)
        static_cast<float *>(row)[j] = v;
    else if constexpr (DT == MOEQ_BF16)
        static_cast<uint16_t *>(row)[j] = (uint16_t)f32_to_bf16_bits(v);
    else
        static_cast<uint16_t *>(row)[j] = __half_as_ushort(__float2half_rn(v));
}

// An integer that orders as the float does (-0 = +0); 0 for NaN, which ranks
// below -inf (kNegInfKey).
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
    if (x != x) return 0u;
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float exp_diff(float x, float m) {
    return f2_lo(exp_neg2(__fadd_rn(x, -m), 0.0f));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// The denominator of the plain weights: sum over the row of exp(x - m), NaN
// where the row holds a NaN or m is +inf (m finite otherwise).
template <int NV>
__device__ __forceinline__ float row_total(const float (&x)[NV], float m) {
    float t = 0.0f;
    bool nan = m == __int_as_float(0x7F800000);
#pragma unroll
    for (int i = 0; i < NV; i += 2) {
        if constexpr (NV == 1) {
            t = exp_diff(x[0], m);
            nan |= x[0] != x[0];
        } else {
            const F2 e = exp_neg2(__fadd_rn(x[i], -m), __fadd_rn(x[i + 1], -m));
            t = __fadd_rn(t, __fadd_rn(f2_lo(e), f2_hi(e)));
            nan |= x[i] != x[i] || x[i + 1] != x[i + 1];
        }
    }
    t = warp_sum(t);
    return __any_sync(0xFFFFFFFFu, nan) ? __int_as_float(0x7FFFFFFF) : t;
}

struct GateParams {
    const uint8_t *logits;
    int64_t stride;  // bytes
    int64_t num_tokens;
    int E, top_k;
    int normalize;
    float scale;
    int32_t *ids;
    float *weights;        // forward
    const float *d_weights;  // gradient
    uint8_t *d_logits;
    uint32_t *err;
};

// Logits j = 32 i + lane of a row; -inf past its end.
template <int DT, int NV>
__device__ __forceinline__ void load_row(const GateParams &p, int64_t t, int lane, float (&x)[NV]) {
    const uint8_t *row = p.logits + t * p.stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = 32 * i + lane;
        x[i] = j < p.E ? load_logit<DT>(row, j) : __int_as_float(0xFF800000);
    }
}

template <int DT, int NV>
__global__ void __launch_bounds__(kGateWarps * 32) gate_kernel(GateParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5);
    if (t >= p.num_tokens) return;
    float x[NV];
    load_row<DT>(p, t, lane, x);
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = order_key(x[i]);
    int my_id = -1;          // lane r: choice r
    uint32_t my_key = 0u, top = 0u;
    for (int r = 0; r < p.top_k; ++r) {
        uint32_t best = 0u;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] > best) {
                best = key[i];
                bi = i;
            }
        const uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, best);
        if (r == 0) top = mx;
        if (mx <= kNegInfKey) break;  // nothing left to choose
        const int j = (int)__reduce_min_sync(0xFFFFFFFFu, best == mx ? 32u * bi + lane : 0xFFFFFFFFu);
        if (lane == r) {
            my_id = j;
            my_key = mx;
        }
        if (lane == (j & 31)) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i == j >> 5) key[i] = 0u;
        }
    }
    float w = 0.0f;
    if (top > kNegInfKey) {
        const float m = key_value(top);
        const float e = my_id >= 0 ? exp_diff(key_value(my_key), m) : 0.0f;
        float total = row_total(x, m);
        if (p.normalize && total == total) total = warp_sum(e);
        if (my_id >= 0 || total != total) w = __fmul_rn(__fdiv_rn(e, total), p.scale);
    }
    if (lane < p.top_k) {
        p.ids[t * p.top_k + lane] = my_id;
        p.weights[t * p.top_k + lane] = w;
    }
}

template <int DT, int NV>
__global__ void __launch_bounds__(kGateWarps * 32) gate_grad_kernel(GateParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5);
    if (t >= p.num_tokens) return;
    float x[NV];
    load_row<DT>(p, t, lane, x);
    float m = __int_as_float(0xFF800000);
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const bool some = m > __int_as_float(0xFF800000);
    int id = -1;
    float d = 0.0f, e = 0.0f;  // lane r: s d_w_r and exp(x_{i_r} - m) of choice r
    if (lane < p.top_k) {
        id = p.ids[t * p.top_k + lane];
        if (id < -1 || id >= p.E) {
            set_error(p.err, MOEQ_DEVERR_BAD_EXPERT);
            id = -1;
        }
        if (id >= 0) d = __fmul_rn(p.d_weights[t * p.top_k + lane], p.scale);
        if (id >= 0 && some) e = exp_diff(load_logit<DT>(p.logits + t * p.stride, id), m);
    }
    float g[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) g[i] = 0.0f;
    if (some) {
        float total = row_total(x, m);
        if (p.normalize && total == total) total = warp_sum(e);
        const float inv = __fdiv_rn(1.0f, total);
        const float q = __fmul_rn(e, inv);
        const float mean = warp_sum(id >= 0 ? __fmul_rn(q, d) : 0.0f);
        if (!p.normalize) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                g[i] = __fmul_rn(-mean, __fmul_rn(exp_diff(x[i], m), inv));
        }
        // the chosen: s q d_w in the plain form (the mean is in already)
        const float add = p.normalize ? __fmul_rn(q, __fadd_rn(d, -mean)) : __fmul_rn(q, d);
        for (int r = 0; r < p.top_k; ++r) {
            const int j = __shfl_sync(0xFFFFFFFFu, id, r);
            const float a = __shfl_sync(0xFFFFFFFFu, add, r);
            if (j < 0 || lane != (j & 31)) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i == j >> 5) g[i] = __fadd_rn(g[i], a);
        }
    }
    uint8_t *row = p.d_logits + t * p.E * (DT == MOEQ_FP32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = 32 * i + lane;
        if (j < p.E) store_logit<DT>(row, j, g[i]);
    }
}

template <int DT>
cudaError_t run_gate(bool grad, const GateParams &p, cudaStream_t s) {
    const unsigned blocks = (unsigned)((p.num_tokens + kGateWarps - 1) / kGateWarps);
    const int nv = (p.E + 31) / 32;
    void (*kern)(GateParams) =
        nv <= 1    ? (grad ? gate_grad_kernel<DT, 1> : gate_kernel<DT, 1>)
        : nv <= 2  ? (grad ? gate_grad_kernel<DT, 2> : gate_kernel<DT, 2>)
        : nv <= 4  ? (grad ? gate_grad_kernel<DT, 4> : gate_kernel<DT, 4>)
        : nv <= 8  ? (grad ? gate_grad_kernel<DT, 8> : gate_kernel<DT, 8>)
        : nv <= 16 ? (grad ? gate_grad_kernel<DT, 16> : gate_kernel<DT, 16>)
                   : (grad ? gate_grad_kernel<DT, 32> : gate_kernel<DT, 32>);
    return launch_pdl(kern, blocks, kGateWarps * 32, 0, s, p);
}

}  // namespace

cudaError_t launch_gate(const GateArgs &a, cudaStream_t s) {
    const int64_t size = a.dtype == MOEQ_FP32 ? 4 : 2;
    GateParams p{static_cast<const uint8_t *>(a.logits), a.stride * size, a.num_tokens,
                 a.num_experts, a.top_k, a.normalize, a.scale, a.ids, a.weights, a.d_weights,
                 static_cast<uint8_t *>(a.d_logits), a.err};
    const bool grad = a.d_logits != nullptr;
    if (a.dtype == MOEQ_BF16) return run_gate<MOEQ_BF16>(grad, p, s);
    if (a.dtype == MOEQ_FP16) return run_gate<MOEQ_FP16>(grad, p, s);
    return run_gate<MOEQ_FP32>(grad, p, s);
}

}  // namespace moeq
