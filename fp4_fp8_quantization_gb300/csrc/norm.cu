// The residual's addition with the root-mean-square norm, an output in 8 bits
// with scales, and the gradient:
//
//   h = x + r (rounded to the stream's type),  u = 1 / sqrt(mean h^2 + eps)
//   y = (h u) w, rounded to the type and / or quantized from fp32 with one scale
//   for each 128 elements or for each row
//
//   with g = w d_y:  d_x = u g - h u^3 mean(g h) + d_h,  d_w = sum over rows of d_y h u
//
// A row is in the registers of the threads of its slot of a CTA, read once:
// thread i holds the vectors i, i + threads, .. of 8 elements, so that 16 lanes
// hold a block of 128.  Sums are fp32 in a fixed order (a thread's elements, the
// lanes of a warp, the warps of a row).
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "fp8_block.cuh"
#include "launch.h"

namespace moeq {

namespace {

// Threads of a row at most: with four vectors a thread, rows past 8192 elements take
// up to 512 threads of 128 registers, all others 256 threads of 255.
constexpr int kMaxThreads = 512;

// 8 consecutive elements as they lie in memory.
template <int DT>
struct Vec8 {
    uint4 u[DT == MOEQ_FP32 ? 2 : 1];
    // outputs may lie over inputs, so not through the read-only path
    __device__ __forceinline__ void load(const void *base, int64_t at) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) +
                                                         at * (DT == MOEQ_FP32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (DT == MOEQ_FP32 ? 2 : 1); ++i)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(u[i].x), "=r"(u[i].y), "=r"(u[i].z), "=r"(u[i].w)
                         : "l"(p + i)
                         : "memory");
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (DT == MOEQ_FP32 ? 2 : 1); ++i) u[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        if constexpr (DT == MOEQ_BF16) {
            unpack8(u[0], x);
        } else if constexpr (DT == MOEQ_FP32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[4 * i] = __uint_as_float(u[i].x);
                x[4 * i + 1] = __uint_as_float(u[i].y);
                x[4 * i + 2] = __uint_as_float(u[i].z);
                x[4 * i + 3] = __uint_as_float(u[i].w);
            }
        } else {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __half2float(__ushort_as_half((unsigned short)(w[i] & 0xFFFFu)));
                x[2 * i + 1] = __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
            }
        }
    }
    // rounded to nearest even
    __device__ __forceinline__ void set(const float (&x)[8]) {
        if constexpr (DT == MOEQ_FP32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                u[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                  __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == MOEQ_BF16)
                    w[i] = f32_to_bf16_bits(x[2 * i]) | (f32_to_bf16_bits(x[2 * i + 1]) << 16);
                else
                    w[i] = (uint32_t)__half_as_ushort(__float2half_rn(x[2 * i])) |
                           ((uint32_t)__half_as_ushort(__float2half_rn(x[2 * i + 1])) << 16);
            }
            u[0] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    // at an element of the buffer of `size` elements
    __device__ __forceinline__ void store(void *base, int64_t at, int64_t size,
                                          uint32_t *err) const {
        constexpr int64_t kS = DT == MOEQ_FP32 ? 4 : 2;
        uint8_t *out = static_cast<uint8_t *>(base) + at * kS;
        if (!store_fits(out, 8 * kS, base, size * kS, err)) return;
#pragma unroll
        for (int i = 0; i < (DT == MOEQ_FP32 ? 2 : 1); ++i)
            st_global_v4(out + 16 * i, u[i].x, u[i].y, u[i].z, u[i].w);
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// The sum or maximum of a value over the `warps` warps of a slot, in every one of its
// threads; part: 32 floats of the CTA, not in use by a reduction before.  Every thread
// of the CTA calls it.
template <bool MAX>
__device__ __forceinline__ float slot_reduce(float v, int warps, float *part) {
    v = MAX ? warp_max(v) : warp_sum(v);
    if (warps == 1) return v;
    const int warp = threadIdx.x >> 5, first = warp / warps * warps;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    float r = part[first];
    for (int i = 1; i < warps; ++i)
        r = MAX ? fmaxf(r, part[first + i]) : __fadd_rn(r, part[first + i]);
    return r;
}

struct NormParams {
    const void *x, *res, *w;
    int64_t x_stride, res_stride, rows;
    int K, threads;  // of a row
    float eps;
    void *h, *y;
    uint8_t *q;
    float *scales;
    int row_scales;
    float *rstd;
    uint32_t *err;
};

template <int DT, int V, int MOST>
__global__ void __launch_bounds__(MOST) norm_kernel(NormParams p) {
    __shared__ float part[2][32];
    pdl_wait();
    pdl_trigger();
    const int warps = p.threads >> 5, i0 = (int)threadIdx.x % p.threads;
    const int64_t slot = (int64_t)blockIdx.x * (blockDim.x / p.threads) + threadIdx.x / p.threads;
    const bool active = slot < p.rows;
    const int64_t t = active ? slot : p.rows - 1;
    Vec8<DT> in[V], res[V], wv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int k = (v * p.threads + i0) * 8;
        if (k < p.K) {
            in[v].load(p.x, t * p.x_stride + k);
            if (p.res) res[v].load(p.res, t * p.res_stride + k);
            wv[v].load(p.w, k);
        } else {
            in[v].zero();
            res[v].zero();
            wv[v].zero();
        }
    }
    float h[V][8], sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int k = (v * p.threads + i0) * 8;
        in[v].values(h[v]);
        if (p.res) {
            float r[8];
            res[v].values(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[v][i] = __fadd_rn(h[v][i], r[i]);
            in[v].set(h[v]);
            in[v].values(h[v]);
            if (active && k < p.K) in[v].store(p.h, t * p.K + k, p.rows * p.K, p.err);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __fmaf_rn(h[v][i], h[v][i], sum);
    }
    sum = slot_reduce<false>(sum, warps, part[0]);
    const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)p.K), p.eps)));
    if (p.rstd && active && i0 == 0) {
        float *out = p.rstd + t;
        if (store_fits(out, 4, p.rstd, p.rows * 4, p.err)) *out = rstd;
    }
    float amax = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int k = (v * p.threads + i0) * 8;
        float w[8];
        wv[v].values(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = __fmul_rn(__fmul_rn(h[v][i], rstd), w[i]);
        if (p.y && active && k < p.K) {
            in[v].set(h[v]);
            in[v].store(p.y, t * p.K + k, p.rows * p.K, p.err);
        }
        if (p.row_scales) amax = fmaxf(amax, amax8(h[v]));
    }
    if (!p.q) return;
    const int64_t KB = p.row_scales ? 1 : (p.K + 127) / 128;
    float s = 0.0f, r = 0.0f;
    if (p.row_scales) {
        s = block_scale(slot_reduce<true>(amax, warps, part[1]));
        r = __fdiv_rn(1.0f, s);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int k = (v * p.threads + i0) * 8;
        if (!p.row_scales) {
            float m = amax8(h[v]);
#pragma unroll
            for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            s = block_scale(m);
            r = __fdiv_rn(1.0f, s);
        }
        if (!active || k >= p.K) continue;
        uint8_t *out = p.q + t * p.K + k;
        if (store_fits(out, 8, p.q, p.rows * p.K, p.err))
            *reinterpret_cast<uint2 *>(out) = codes8(h[v], r);
        float *scale = p.scales + t * KB + (p.row_scales ? 0 : k / 128);
        if ((p.row_scales ? k == 0 : (i0 & 15) == 0) &&
            store_fits(scale, 4, p.scales, p.rows * KB * 4, p.err))
            *scale = s;
    }
}

struct NormGradParams {
    const void *dy, *dh, *h, *w;
    int64_t dy_stride, dh_stride, h_stride, rows;
    const float *rstd;
    int K, threads;
    void *dx;
    float *part;  // [slots of the grid][K] sums of the weight's gradient, or null
    uint32_t *err;
};

template <int DT, int V, int MOST>
__global__ void __launch_bounds__(MOST) norm_grad_kernel(NormGradParams p) {
    __shared__ float part[2][32];
    pdl_wait();
    pdl_trigger();
    const int warps = p.threads >> 5, i0 = (int)threadIdx.x % p.threads;
    const int slots = blockDim.x / p.threads;
    const int64_t slot = (int64_t)blockIdx.x * slots + threadIdx.x / p.threads;
    float dw[V][8];
    Vec8<DT> wv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int k = (v * p.threads + i0) * 8;
        wv[v].zero();
        if (k < p.K) wv[v].load(p.w, k);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    }
    // every slot of the CTA walks the same number of rows: they share its barriers
    const int64_t step = (int64_t)gridDim.x * slots;
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * slots; t0 < p.rows; t0 += step, turn ^= 1) {
        const int64_t row = t0 + (slot - (int64_t)blockIdx.x * slots);
        const bool active = row < p.rows;
        const int64_t t = active ? row : p.rows - 1;
        Vec8<DT> hv[V], gv[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int k = (v * p.threads + i0) * 8;
            hv[v].zero();
            gv[v].zero();
            if (k < p.K && active) {
                hv[v].load(p.h, t * p.h_stride + k);
                gv[v].load(p.dy, t * p.dy_stride + k);
            }
        }
        const float u = __ldg(p.rstd + t);
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float h[8], g[8], w[8];
            hv[v].values(h);
            gv[v].values(g);
            wv[v].values(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[v][i] = __fmaf_rn(g[i], __fmul_rn(h[i], u), dw[v][i]);
                dot = __fmaf_rn(__fmul_rn(g[i], w[i]), h[i], dot);
            }
        }
        dot = slot_reduce<false>(dot, warps, part[turn]);
        // d_x = u (g w - h mean(g w h) u^2)
        const float back = __fmul_rn(__fdiv_rn(dot, (float)p.K), __fmul_rn(u, u));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int k = (v * p.threads + i0) * 8;
            if (!active || k >= p.K) continue;
            float h[8], g[8], w[8];
            hv[v].values(h);
            gv[v].values(g);
            wv[v].values(w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[i] = __fmul_rn(__fmaf_rn(-h[i], back, __fmul_rn(g[i], w[i])), u);
            if (p.dh) {
                float d[8];
                hv[v].load(p.dh, t * p.dh_stride + k);
                hv[v].values(d);
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = __fadd_rn(g[i], d[i]);
            }
            hv[v].set(g);
            hv[v].store(p.dx, t * p.K + k, p.rows * p.K, p.err);
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int k = (v * p.threads + i0) * 8;
        if (k >= p.K) continue;
        uint8_t *out = reinterpret_cast<uint8_t *>(p.part + slot * p.K + k);
        if (!store_fits(out, 32, p.part, step * p.K * 4, p.err)) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            st_global_v4(out + 16 * i, __float_as_uint(dw[v][4 * i]),
                         __float_as_uint(dw[v][4 * i + 1]), __float_as_uint(dw[v][4 * i + 2]),
                         __float_as_uint(dw[v][4 * i + 3]));
    }
}

// The sums of `parts` rows of K partial sums: 32 columns a CTA, its warps take every
// 32nd row and join.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float *part, int parts, int K,
                                                         float *out, uint32_t *err) {
    __shared__ float sums[32][33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int k = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (k < K)
        for (int r = warp; r < parts; r += 32) v = __fadd_rn(v, __ldg(part + (int64_t)r * K + k));
    sums[warp][lane] = v;
    __syncthreads();
    v = warp_sum(sums[lane][warp]);
    const int at = blockIdx.x * 32 + warp;
    if (lane == 0 && at < K) {
        float *o = out + at;
        if (store_fits(o, 4, out, (int64_t)K * 4, err)) *o = v;
    }
}

// Threads of a row and vectors of each.
struct Split {
    int v, threads, slots;  // slots: rows of a CTA
};

Split split_of(int64_t K) {
    const int vecs = (int)((K + 7) / 8);
    int v = 1;
    while (v < 4 && (vecs + v - 1) / v > 256) v *= 2;
    const int threads = ((vecs + v - 1) / v + 31) / 32 * 32;
    return {v, threads, std::max(1, 128 / threads)};
}

template <int DT, int V, int MOST = 256>
cudaError_t run_norm(const NormParams &p, const Split &c, cudaStream_t s) {
    return launch_pdl(norm_kernel<DT, V, MOST>, (unsigned)((p.rows + c.slots - 1) / c.slots),
                      c.threads * c.slots, 0, s, p);
}

template <int DT>
cudaError_t run_norm_type(NormParams p, cudaStream_t s) {
    const Split c = split_of(p.K);
    p.threads = c.threads;
    return c.v == 1 ? run_norm<DT, 1>(p, c, s)
           : c.v == 2 ? run_norm<DT, 2>(p, c, s)
           : c.threads <= 256 ? run_norm<DT, 4>(p, c, s)
                              : run_norm<DT, 4, kMaxThreads>(p, c, s);
}

// The gradient's grid: as many rows in flight as two CTAs on each SM of this
// machine have, fewer where there are fewer rows.  It depends on the sizes
// alone, so that the workspace's size does.
int grad_ctas(int64_t rows, const Split &c) {
    return (int)std::min<int64_t>((rows + c.slots - 1) / c.slots, 2 * 152);
}

template <int DT, int V, int MOST = 256>
cudaError_t run_grad(const NormGradParams &p, const Split &c, cudaStream_t s) {
    return launch_pdl(norm_grad_kernel<DT, V, MOST>, (unsigned)grad_ctas(p.rows, c), c.threads * c.slots,
                      0, s, p);
}

template <int DT>
cudaError_t run_grad_type(NormGradParams p, cudaStream_t s) {
    const Split c = split_of(p.K);
    p.threads = c.threads;
    return c.v == 1 ? run_grad<DT, 1>(p, c, s)
           : c.v == 2 ? run_grad<DT, 2>(p, c, s)
           : c.threads <= 256 ? run_grad<DT, 4>(p, c, s)
                              : run_grad<DT, 4, kMaxThreads>(p, c, s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, cudaStream_t s) {
    const NormParams p{a.x, a.res, a.w, a.x_stride, a.res_stride, a.rows, (int)a.K, 0,
                       a.eps, a.h, a.y, a.q, a.scales, a.row_scales, a.rstd, a.err};
    if (a.dtype == MOEQ_BF16) return run_norm_type<MOEQ_BF16>(p, s);
    if (a.dtype == MOEQ_FP16) return run_norm_type<MOEQ_FP16>(p, s);
    return run_norm_type<MOEQ_FP32>(p, s);
}

int64_t norm_grad_parts(int64_t rows, int64_t K) {
    if (rows == 0) return 0;
    const Split c = split_of(K);
    return (int64_t)grad_ctas(rows, c) * c.slots;
}

cudaError_t launch_norm_grad(const NormGradArgs &a, cudaStream_t s) {
    const NormGradParams p{a.dy, a.dh, a.h, a.w, a.dy_stride, a.dh_stride, a.h_stride, a.rows,
                           a.rstd, (int)a.K, 0, a.dx, a.d_weight ? a.workspace : nullptr, a.err};
    const cudaError_t e = a.rows == 0            ? cudaSuccess
                          : a.dtype == MOEQ_BF16 ? run_grad_type<MOEQ_BF16>(p, s)
                          : a.dtype == MOEQ_FP16 ? run_grad_type<MOEQ_FP16>(p, s)
                                                 : run_grad_type<MOEQ_FP32>(p, s);
    if (e != cudaSuccess || !a.d_weight) return e;
    return launch_pdl(sum_parts_kernel, (unsigned)((a.K + 31) / 32), 1024, 0, s,
                      (const float *)a.workspace, (int)norm_grad_parts(a.rows, a.K), (int)a.K,
                      a.d_weight, a.err);
}

}  // namespace moeq
