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

// How the pieces of a token are dealt out.
enum Form {
    kPiece,  // one per thread: grid (tokens, shares of a row)
    kFlat,   // one per thread of a flat grid, for short rows
    kCta,    // a CTA per token, with the dots of the weights' gradient
    kWarp    // a warp per token with the dots, for short rows
};

struct Place {
    int64_t t, at, step;  // token, first byte and stride of the thread's pieces
};

template <int FORM>
__device__ __forceinline__ Place my_place(const RowsParams &p) {
    if constexpr (FORM == kPiece)
        return {(int64_t)blockIdx.x, ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 16,
                p.row_bytes};
    if constexpr (FORM == kFlat) {  // the host keeps tokens * pieces below 2^32
        const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
        const uint32_t pieces = (uint32_t)(p.row_bytes >> 4), t = i / pieces;
        return {(int64_t)t, (int64_t)(i - t * pieces) * 16, p.row_bytes};
    }
    if constexpr (FORM == kCta)
        return {(int64_t)blockIdx.x, (int64_t)threadIdx.x * 16, (int64_t)blockDim.x * 16};
    return {(int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5),
            (int64_t)(threadIdx.x & 31) * 16, 512};
}

__device__ __forceinline__ void store_dot(const RowsParams &p, int64_t choice, float v) {
    if (store_fits(p.dw + choice, 4, p.dw, p.num_tokens * p.top_k * 4, p.err)) p.dw[choice] = v;
}

// The KC dot products of a token's threads, summed and stored in d_w.  Every
// thread of the token calls it; the order of the sum is fixed by their number.
template <int FORM, int KC>
__device__ __forceinline__ void store_dots(const RowsParams &p, int64_t t, float (&s)[KC]) {
#pragma unroll
    for (int j = 0; j < KC; ++j)
#pragma unroll
        for (int o = 16; o; o >>= 1) s[j] = __fadd_rn(s[j], __shfl_xor_sync(0xFFFFFFFFu, s[j], o));
    const int lane = threadIdx.x & 31;
    if constexpr (FORM == kWarp) {
#pragma unroll
        for (int j = 0; j < KC; ++j)
            if (lane == j && j < p.top_k) store_dot(p, t * p.top_k + j, s[j]);
    } else {
        __shared__ float part[4][KC];
        if (lane == 0) {
#pragma unroll
            for (int j = 0; j < KC; ++j) part[threadIdx.x >> 5][j] = s[j];
        }
        __syncthreads();
        if ((int)threadIdx.x < p.top_k) {
            float v = 0.0f;
            for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v = __fadd_rn(v, part[i][threadIdx.x]);
            store_dot(p, t * p.top_k + threadIdx.x, v);
        }
    }
}

// Token -> rows.  With dots (top_k <= KC) the rows that they read are loaded
// KC at a time, so that a token and its rows are each touched once.
template <int DT, int KC, int FORM>
__global__ void __launch_bounds__(160) spread_kernel(RowsParams p) {
    constexpr bool DOTS = FORM == kCta || FORM == kWarp;
    pdl_wait();
    pdl_trigger();
    const Place me = my_place<FORM>(p);
    if (me.t >= p.num_tokens) return;  // a whole warp, or no dots
    float dot[KC] = {};
    for (int j0 = 0; j0 < (DOTS ? KC : p.top_k); j0 += KC) {
        Choices<KC> ch;
        ch.load(p, me.t, j0, me.at == 0);
        for (int64_t a = me.at; a < p.row_bytes; a += me.step) {
            uint4 y[DOTS ? KC : 1];
            if constexpr (DOTS) {
#pragma unroll
                for (int j = 0; j < KC; ++j)
                    if (ch.row[j] >= 0) y[j] = ld_stream(p.rows_in + ch.row[j] + a);
            }
            const uint4 u = *reinterpret_cast<const uint4 *>(p.token_in + me.t * p.token_stride + a);
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
                uint8_t *out = p.rows_out + ch.row[j] + a;
                if (store_fits(out, 16, p.rows_out, p.total_rows * p.row_bytes, p.err))
                    *reinterpret_cast<uint4 *>(out) = o;
                if constexpr (DOTS) {
                    Vec<DT> v;
                    v.from(y[j]);
#pragma unroll
                    for (int i = 0; i < Vec<DT>::N; ++i) dot[j] = __fmaf_rn(x.v[i], v.v[i], dot[j]);
                }
            }
        }
    }
    if constexpr (DOTS) store_dots<FORM, KC>(p, me.t, dot);
}

// Rows -> token; KC rows are in flight at a time.
template <int DT, int KC, int FORM>
__global__ void __launch_bounds__(160) collect_kernel(RowsParams p) {
    constexpr bool DOTS = FORM == kCta || FORM == kWarp;
    pdl_wait();
    pdl_trigger();
    const Place me = my_place<FORM>(p);
    if (me.t >= p.num_tokens) return;  // a whole warp, or no dots
    float dot[KC] = {};
    Choices<KC> ch;
    ch.load(p, me.t, 0, me.at == 0);
    for (int64_t a = me.at; a < p.row_bytes; a += me.step) {
        Vec<DT> acc, x;
#pragma unroll
        for (int i = 0; i < Vec<DT>::N; ++i) acc.v[i] = 0.0f;
        if constexpr (DOTS)
            x.from(*reinterpret_cast<const uint4 *>(p.token_in + me.t * p.token_stride + a));
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
            ch.load(p, me.t, j0, me.at == 0);  // one piece per thread: read once
        }
        uint8_t *out = p.token_out + me.t * p.row_bytes + a;
        if (store_fits(out, 16, p.token_out, p.num_tokens * p.row_bytes, p.err))
            *reinterpret_cast<uint4 *>(out) = acc.pack();
    }
    if constexpr (DOTS) store_dots<FORM, KC>(p, me.t, dot);
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
    if (lane == 0) store_dot(p, c, s);
}

// Threads of a CTA for rows of `pieces` pieces: the first of the sizes that
// leaves the fewest threads of a row's last share without a piece.  Small CTAs
// whose shares fill them are the faster ones (16384 tokens, top-8, 4096 bf16:
// collect 182 us with 128 threads, 204 with 256; with dots, two thirds idle in
// the last share of 320 pieces, 63 us against 51), but one-piece CTAs below 96
// threads are bound by their launch rate (320 pieces: 83 us with 64, 44 with
// 160).
unsigned cta_threads(int64_t pieces, const int (&sizes)[3]) {
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

template <int DT, int KC, int FORM>
cudaError_t launch_rows(bool spread, dim3 grid, unsigned threads, const RowsParams &p,
                        cudaStream_t s) {
    return launch_pdl(spread ? spread_kernel<DT, KC, FORM> : collect_kernel<DT, KC, FORM>, grid,
                      threads, 0, s, p);
}

template <int DT, int KC>
cudaError_t run_rows(bool spread, const RowsParams &p, cudaStream_t s) {
    const int64_t pieces = p.row_bytes / 16, T = p.num_tokens;
    // several tokens per CTA for rows that would leave one mostly empty: top-4
    // of 15769 x 112 fp16 33 -> 13 us forward and gradient
    const bool shorts = pieces < 96;
    if (p.dw && p.top_k <= KC) {
        if (shorts) return launch_rows<DT, KC, kWarp>(spread, (unsigned)((T + 3) / 4), 128, p, s);
        return launch_rows<DT, KC, kCta>(spread, (unsigned)T, cta_threads(pieces, {128, 96, 64}),
                                         p, s);
    }
    cudaError_t e;
    if (shorts && T * pieces < (int64_t)1 << 32) {
        e = launch_rows<DT, KC, kFlat>(spread, (unsigned)((T * pieces + 127) / 128), 128, p, s);
    } else {
        const unsigned threads = cta_threads(pieces, {128, 160, 96});
        e = launch_rows<DT, KC, kPiece>(
            spread, dim3((unsigned)T, (unsigned)((pieces + threads - 1) / threads)), threads, p, s);
    }
    if (e != cudaSuccess || !p.dw) return e;
    // more choices than KC: the dots apart, which read the rows and, once for each
    // choice, the token (bf16, 8192 x 4096: permute's gradient 107 us for top-8,
    // 220 for top-9, 99 and 109 of memory; combine's 174 and 211, 168 and 188)
    const int64_t choices = T * p.top_k;
    return launch_pdl(dots_kernel<DT>, (unsigned)((choices + 3) / 4), 128, 0, s, p);
}

template <int DT>
cudaError_t run_rows(bool spread, const RowsParams &p, cudaStream_t s) {
    if (p.top_k <= 2) return run_rows<DT, 2>(spread, p, s);
    if (p.top_k <= 4) return run_rows<DT, 4>(spread, p, s);
    return run_rows<DT, 8>(spread, p, s);
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
