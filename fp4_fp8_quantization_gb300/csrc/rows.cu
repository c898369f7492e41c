// Tokens to their experts' rows and back, with the router's weights, and the
// gradients of both.  dst[t, j] is the row of choice j of token t (from
// moeq_route_topk; -1 for a dropped choice), w its weight:
//
//   permute   rows[dst[t, j]] = w[t, j] x[t]
//             d_x[t] = sum_j w[t, j] d_rows[dst[t, j]]
//             d_w[t, j] = <x[t], d_rows[dst[t, j]]>
//   combine   y[t] = sum_j w[t, j] rows[dst[t, j]]
//             d_rows[dst[t, j]] = w[t, j] d_y[t]
//             d_w[t, j] = <d_y[t], rows[dst[t, j]]>
//
// The gradient of each is the other with the dot products of d_w, so two
// kernels do all four: spread_kernel (token -> rows) and collect_kernel
// (rows -> token), each with or without the dots.  Both run token by token:
// a token is read or written once, its k rows are whole contiguous rows, and
// the sums over j are taken by one thread in the order of j (no atomics: the
// results do not depend on the launch).  Products and sums are held in fp32
// and rounded once when stored; without weights rows are copied as bits.
#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.h"

namespace moeq {

namespace {

// 16 bytes of a row as fp32 values (element type DT: moeq_dtype).
template <int DT>
struct Vec {
    static constexpr int N = DT == MOEQ_FP32 ? 4 : 8;
    float v[N];
    __device__ __forceinline__ void from(const uint4 &u) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == MOEQ_FP32) {
                v[i] = __uint_as_float(w[i]);
            } else if constexpr (DT == MOEQ_BF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
    // rounded to nearest even
    __device__ __forceinline__ uint4 pack() const {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == MOEQ_FP32) {
                w[i] = __float_as_uint(v[i]);
            } else if constexpr (DT == MOEQ_BF16) {
                w[i] = f32_to_bf16_bits(v[2 * i]) | (f32_to_bf16_bits(v[2 * i + 1]) << 16);
            } else {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct RowsParams {
    const uint8_t *token_in;   // spread: the tokens; collect: the dots' tokens (or null)
    int64_t token_stride;      // bytes
    uint8_t *token_out;        // collect: [num_tokens, H]
    const uint8_t *rows_in;    // collect: the rows; spread: the dots' rows (or null)
    uint8_t *rows_out;         // spread
    const int32_t *dst;
    const float *w;            // null: 1
    float *dw;                 // null: no dots
    int64_t num_tokens, total_rows;
    int64_t row_bytes;
    int top_k;
    uint32_t *err;
};

// The row of choice c, -1 if it was dropped (or, with an error, is no row).
__device__ __forceinline__ int64_t row_of(const RowsParams &p, int64_t c, bool report) {
    const int r = __ldg(p.dst + c);
    if (r >= 0 && r < p.total_rows) return r;
    if (r != -1 && report) set_error(p.err, MOEQ_DEVERR_BAD_INDEX);
    return -1;
}

// One 16-byte piece of one token per thread: grid (pieces / threads, tokens).
template <int DT>
__global__ void __launch_bounds__(128) spread_kernel(RowsParams p) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int64_t at = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 16;
    if (at >= p.row_bytes) return;
    const uint4 u = *reinterpret_cast<const uint4 *>(p.token_in + t * p.token_stride + at);
    Vec<DT> x;
    x.from(u);
    for (int j = 0; j < p.top_k; ++j) {
        const int64_t c = t * p.top_k + j;
        const int64_t r = row_of(p, c, at == 0);
        if (r < 0) continue;
        uint4 o = u;
        if (p.w) {
            const float w = __ldg(p.w + c);
            Vec<DT> y;
#pragma unroll
            for (int i = 0; i < Vec<DT>::N; ++i) y.v[i] = __fmul_rn(x.v[i], w);
            o = y.pack();
        }
        *reinterpret_cast<uint4 *>(p.rows_out + r * p.row_bytes + at) = o;
    }
}

template <int DT>
__global__ void __launch_bounds__(128) collect_kernel(RowsParams p) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int64_t at = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 16;
    if (at >= p.row_bytes) return;
    Vec<DT> acc;
#pragma unroll
    for (int i = 0; i < Vec<DT>::N; ++i) acc.v[i] = 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
        const int64_t c = t * p.top_k + j;
        const int64_t r = row_of(p, c, at == 0);
        if (r < 0) continue;
        const float w = p.w ? __ldg(p.w + c) : 1.0f;
        Vec<DT> x;
        x.from(*reinterpret_cast<const uint4 *>(p.rows_in + r * p.row_bytes + at));
#pragma unroll
        for (int i = 0; i < Vec<DT>::N; ++i) acc.v[i] = __fmaf_rn(x.v[i], w, acc.v[i]);
    }
    *reinterpret_cast<uint4 *>(p.token_out + t * p.row_bytes + at) = acc.pack();
}

// d_w[t, j] = <token_in[t], rows_in[dst[t, j]]>: one warp per choice, 0 for a
// dropped one.
template <int DT>
__global__ void __launch_bounds__(128) dots_kernel(RowsParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (c >= p.num_tokens * p.top_k) return;
    const int64_t r = row_of(p, c, false);
    float s = 0.0f;
    if (r >= 0) {
        const uint8_t *a = p.token_in + c / p.top_k * p.token_stride, *b = p.rows_in + r * p.row_bytes;
        for (int64_t at = lane * 16; at < p.row_bytes; at += 512) {
            Vec<DT> x, y;
            x.from(*reinterpret_cast<const uint4 *>(a + at));
            y.from(*reinterpret_cast<const uint4 *>(b + at));
#pragma unroll
            for (int i = 0; i < Vec<DT>::N; ++i) s = __fmaf_rn(x.v[i], y.v[i], s);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
    if (lane == 0) p.dw[c] = s;
}

template <int DT>
cudaError_t run_rows(bool spread, const RowsParams &p, cudaStream_t s) {
    const int64_t pieces = p.row_bytes / 16;
    const dim3 grid((unsigned)p.num_tokens, (unsigned)((pieces + 127) / 128));
    cudaError_t e = spread ? launch_pdl(spread_kernel<DT>, grid, 128, 0, s, p)
                           : launch_pdl(collect_kernel<DT>, grid, 128, 0, s, p);
    if (e != cudaSuccess || !p.dw) return e;
    const int64_t choices = p.num_tokens * p.top_k;
    return launch_pdl(dots_kernel<DT>, (unsigned)((choices + 3) / 4), 128, 0, s, p);
}

}  // namespace

cudaError_t launch_topk_rows(const RowsArgs &a, cudaStream_t s) {
    const int64_t size = a.dtype == MOEQ_FP32 ? 4 : 2;
    RowsParams p{static_cast<const uint8_t *>(a.token_in), a.token_stride * size,
                 static_cast<uint8_t *>(a.token_out), static_cast<const uint8_t *>(a.rows_in),
                 static_cast<uint8_t *>(a.rows_out), a.dst, a.weights, a.d_weights, a.num_tokens,
                 a.total_rows, a.hidden * size, a.top_k, a.err};
    if (a.dtype == MOEQ_BF16) return run_rows<MOEQ_BF16>(a.spread, p, s);
    if (a.dtype == MOEQ_FP16) return run_rows<MOEQ_FP16>(a.spread, p, s);
    return run_rows<MOEQ_FP32>(a.spread, p, s);
}

}  // namespace moeq
