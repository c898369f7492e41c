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

// The rows of choices j0 .. j0 + KC - 1 of token t (-1: none) and their
// weights.
template <int KC>
struct Choices {
    int64_t row[KC];  // byte offset of the row, < 0 without one
    float w[KC];
    __device__ __forceinline__ void load(const RowsParams &p, int64_t t, int j0, bool report) {
#pragma unroll
        for (int j = 0; j < KC; ++j) {
            const int64_t c = t * p.top_k + j0 + j;
            row[j] = -1;
            w[j] = 1.0f;
            if (j0 + j < p.top_k) {
                const int64_t r = row_of(p, c, report);
                row[j] = r < 0 ? -1 : r * p.row_bytes;
                if (p.w) w[j] = __ldg(p.w + c);
            }
        }
    }
};

// The KC dot products of a CTA's threads, summed and stored in d_w.  Every
// thread calls it; the order of the sum is fixed by the CTA's size.
template <int KC>
__device__ __forceinline__ void store_dots(const RowsParams &p, int64_t t, float (&s)[KC]) {
    __shared__ float part[8][KC];
#pragma unroll
    for (int j = 0; j < KC; ++j)
#pragma unroll
        for (int o = 16; o; o >>= 1) s[j] = __fadd_rn(s[j], __shfl_xor_sync(0xFFFFFFFFu, s[j], o));
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int j = 0; j < KC; ++j) part[threadIdx.x >> 5][j] = s[j];
    }
    __syncthreads();
    if ((int)threadIdx.x < p.top_k) {
        float v = 0.0f;
        for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v = __fadd_rn(v, part[i][threadIdx.x]);
        p.dw[t * p.top_k + threadIdx.x] = v;
    }
}

// Token -> rows.  Without dots: one 16-byte piece of a token per thread, grid
// (tokens, pieces / threads).  With dots (top_k <= KC): one CTA per token; the
// rows that the dots read are loaded KC at a time, so that a token and its
// rows are each touched once.
template <int DT, int KC, bool DOTS>
__global__ void __launch_bounds__(256) spread_kernel(RowsParams p) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    int64_t at = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 16;
    float dot[KC] = {};
    for (int j0 = 0; j0 < (DOTS ? KC : p.top_k); j0 += KC) {
        Choices<KC> ch;
        ch.load(p, t, j0, at == 0);
        for (int64_t a = at; a < p.row_bytes; a += (int64_t)blockDim.x * 16) {
            uint4 y[DOTS ? KC : 1];
            if constexpr (DOTS) {
#pragma unroll
                for (int j = 0; j < KC; ++j)
                    if (ch.row[j] >= 0) y[j] = ld_stream(p.rows_in + ch.row[j] + a);
            }
            const uint4 u = *reinterpret_cast<const uint4 *>(p.token_in + t * p.token_stride + a);
            Vec<DT> x;
            x.from(u);
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                if (ch.row[j] < 0) continue;
                uint4 o = u;
                if (p.w) {
                    Vec<DT> v;
#pragma unroll
                    for (int i = 0; i < Vec<DT>::N; ++i) v.v[i] = __fmul_rn(x.v[i], ch.w[j]);
                    o = v.pack();
                }
                if (store_ok(ch.row[j] + a < p.total_rows * p.row_bytes, p.err))
                    *reinterpret_cast<uint4 *>(p.rows_out + ch.row[j] + a) = o;
                if constexpr (DOTS) {
                    Vec<DT> v;
                    v.from(y[j]);
#pragma unroll
                    for (int i = 0; i < Vec<DT>::N; ++i) dot[j] = __fmaf_rn(x.v[i], v.v[i], dot[j]);
                }
            }
            if (!DOTS) break;  // one piece per thread
        }
    }
    if constexpr (DOTS) store_dots<KC>(p, t, dot);
}

// Rows -> token, in the same two forms; KC rows are in flight at a time.
template <int DT, int KC, bool DOTS>
__global__ void __launch_bounds__(256) collect_kernel(RowsParams p) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int64_t at = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 16;
    float dot[KC] = {};
    Choices<KC> ch;
    ch.load(p, t, 0, at == 0);
    for (int64_t a = at; a < p.row_bytes; a += (int64_t)blockDim.x * 16) {
        Vec<DT> acc, x;
#pragma unroll
        for (int i = 0; i < Vec<DT>::N; ++i) acc.v[i] = 0.0f;
        if constexpr (DOTS)
            x.from(*reinterpret_cast<const uint4 *>(p.token_in + t * p.token_stride + a));
        for (int j0 = 0;;) {
            uint4 y[KC];
#pragma unroll
            for (int j = 0; j < KC; ++j)
                if (ch.row[j] >= 0) y[j] = ld_stream(p.rows_in + ch.row[j] + a);
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                if (ch.row[j] < 0) continue;
                Vec<DT> v;
                v.from(y[j]);
#pragma unroll
                for (int i = 0; i < Vec<DT>::N; ++i) {
                    acc.v[i] = __fmaf_rn(v.v[i], ch.w[j], acc.v[i]);
                    if constexpr (DOTS) dot[j] = __fmaf_rn(x.v[i], v.v[i], dot[j]);
                }
            }
            j0 += KC;
            if (DOTS || j0 >= p.top_k) break;
            ch.load(p, t, j0, at == 0);
        }
        if (store_ok(t < p.num_tokens, p.err))
            *reinterpret_cast<uint4 *>(p.token_out + t * p.row_bytes + a) = acc.pack();
        if (!DOTS) break;  // one piece per thread
    }
    if constexpr (DOTS) store_dots<KC>(p, t, dot);
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

// Threads of a CTA for rows of `pieces` pieces: a whole short row, else the
// first of the sizes that leaves the fewest threads of a row's last share
// without a piece.  Small CTAs whose shares fill them are the faster ones
// (16384 tokens, top-8, 4096 bf16: collect 182 us with 128 threads, 204 with
// 256; with dots, two thirds idle in the last share of 320 pieces, 63 us
// against 51), but one-piece CTAs below 96 threads are bound by their launch
// rate (320 pieces: 83 us with 64, 44 with 160).
unsigned cta_threads(int64_t pieces, const int (&sizes)[3]) {
    if (pieces <= 128) return (unsigned)(pieces + 31) / 32 * 32;
    int best = 0;
    int64_t idle = INT64_MAX;
    for (const int n : sizes) {
        const int64_t rest = (pieces + n - 1) / n * n - pieces;
        if (rest < idle) {
            idle = rest;
            best = n;
        }
    }
    return (unsigned)best;
}

template <int DT, int KC>
cudaError_t run_rows(bool spread, const RowsParams &p, cudaStream_t s) {
    const int64_t pieces = p.row_bytes / 16;
    if (p.dw && p.top_k <= KC)
        return launch_pdl(spread ? spread_kernel<DT, KC, true> : collect_kernel<DT, KC, true>,
                          (unsigned)p.num_tokens, cta_threads(pieces, {128, 96, 64}), 0, s, p);
    const unsigned threads = cta_threads(pieces, {128, 160, 96});
    const dim3 grid((unsigned)p.num_tokens, (unsigned)((pieces + threads - 1) / threads));
    const cudaError_t e = launch_pdl(
        spread ? spread_kernel<DT, KC, false> : collect_kernel<DT, KC, false>, grid, threads, 0, s,
        p);
    if (e != cudaSuccess || !p.dw) return e;
    const int64_t choices = p.num_tokens * p.top_k;  // more choices than KC: the dots apart
    return launch_pdl(dots_kernel<DT>, (unsigned)((choices + 3) / 4), 128, 0, s, p);
}

template <int DT>
cudaError_t run_rows(bool spread, const RowsParams &p, cudaStream_t s) {
    return p.top_k <= 2 ? run_rows<DT, 2>(spread, p, s) : run_rows<DT, 8>(spread, p, s);
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
