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
// lanes of a warp, the warps of a row).  The gradient walks rows with persistent CTAs,
// the weight's sums in registers; each slot leaves one row of them, which a second
// kernel adds.
//
// Bound by memory.  Share of the copy rate: x + residual to h and y, bf16, 16384 x 7168
// 137 us (1.01), 8191 x 4096 41 (0.97), 65536 x 1024 79 (1.01), 131072 x 256 42 (0.94);
// to h and 128-block codes 135 (0.90), 38 (0.92), 70 (0.99), 45 (0.76); fp16 to y and
// codes by rows, a second reduction, 5003 x 2480 14 (0.66).  Gradient with all its
// inputs, 16384 x 7168 159 (0.87), 8191 x 4096 47 (0.85), 65536 x 1024 94 (0.84), fp32
// 8192 x 4096 91 (0.87).  Rows past 8192 elements leave an SM two CTAs or one: 4096 x
// 16384 101 (0.79) and 142 (0.56).
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "fp8_block.cuh"
#include "launch.h"

namespace moeq {

namespace {

// Threads of a row at most.
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
    // of what no call writes, kept in the cache of the SM
    __device__ __forceinline__ void load_kept(const void *base, int64_t at) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) +
                                                         at * (DT == MOEQ_FP32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (DT == MOEQ_FP32 ? 2 : 1); ++i) u[i] = __ldg(p + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (DT == MOEQ_FP32 ? 2 : 1); ++i) u[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void values(F2 (&x)[4]) const {
        if constexpr (DT == MOEQ_FP32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[2 * i] = f2(__uint_as_float(u[i].x), __uint_as_float(u[i].y));
                x[2 * i + 1] = f2(__uint_as_float(u[i].z), __uint_as_float(u[i].w));
            }
        } else {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == MOEQ_BF16) {
                    x[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
                } else {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                    x[i] = f2(v.x, v.y);
                }
            }
        }
    }
    // rounded to nearest even
    __device__ __forceinline__ void set(const F2 (&x)[4]) {
        if constexpr (DT == MOEQ_FP32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                u[i] = make_uint4(__float_as_uint(f2_lo(x[2 * i])), __float_as_uint(f2_hi(x[2 * i])),
                                  __float_as_uint(f2_lo(x[2 * i + 1])),
                                  __float_as_uint(f2_hi(x[2 * i + 1])));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == MOEQ_BF16) {
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                        : "=r"(w[i])
                        : "f"(f2_hi(x[i])), "f"(f2_lo(x[i])));
                } else {
                    const __half2 v = __floats2half2_rn(f2_lo(x[i]), f2_hi(x[i]));
                    w[i] = *reinterpret_cast<const uint32_t *>(&v);
                }
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

// The largest of V vectors' amax over the 16 lanes of each one's block: lane l of them
// gets that of vector l / (16 / V) (each step sends what the other half of the lanes keeps).
template <int V>
__device__ __forceinline__ float blocks_amax(const float (&m)[V], int lane) {
    constexpr unsigned kAll = 0xFFFFFFFFu;
    float k[V];
#pragma unroll
    for (int v = 0; v < V; ++v) k[v] = m[v];
    int o = 8;
#pragma unroll
    for (int n = V / 2; n; n /= 2, o /= 2) {
        const bool upper = lane & o;
#pragma unroll
        for (int v = 0; v < n; ++v)
            k[v] = fmaxf(upper ? k[v + n] : k[v], __shfl_xor_sync(kAll, upper ? k[v] : k[v + n], o));
    }
#pragma unroll
    for (; o; o /= 2) k[0] = fmaxf(k[0], __shfl_xor_sync(kAll, k[0], o));
    return k[0];
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
            wv[v].load_kept(p.w, k);
        } else {
            in[v].zero();
            res[v].zero();
            wv[v].zero();
        }
    }
    F2 h[V][4], sq = f2s(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int k = (v * p.threads + i0) * 8;
        in[v].values(h[v]);
        if (p.res) {
            F2 r[4];
            res[v].values(r);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[v][i] = add2(h[v][i], r[i]);
            in[v].set(h[v]);
            in[v].values(h[v]);
            if (active && k < p.K) in[v].store(p.h, t * p.K + k, p.rows * p.K, p.err);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sq = fma2(h[v][i], h[v][i], sq);
    }
    const float sum = slot_reduce<false>(__fadd_rn(f2_lo(sq), f2_hi(sq)), warps, part[0]);
    const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)p.K), p.eps)));
    if (p.rstd && active && i0 == 0) {
        float *out = p.rstd + t;
        if (store_fits(out, 4, p.rstd, p.rows * 4, p.err)) *out = rstd;
    }
    float amax[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int k = (v * p.threads + i0) * 8;
        F2 w[4];
        wv[v].values(w);
        amax[v] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[v][i] = mul2(mul2(h[v][i], f2s(rstd)), w[i]);
            // fmaxf drops a NaN operand, so a NaN never becomes the amax
            amax[v] = fmaxf(fmaxf(amax[v], fabsf(f2_lo(h[v][i]))), fabsf(f2_hi(h[v][i])));
        }
        if (p.y && active && k < p.K) {
            in[v].set(h[v]);
            in[v].store(p.y, t * p.K + k, p.rows * p.K, p.err);
        }
    }
    if (!p.q) return;
    const int64_t KB = p.row_scales ? 1 : (p.K + 127) / 128;
    // 1 / scale of each vector: one scale for the row, or of the 16 lanes of a block, where
    // a lane takes the quotients of one vector for all
    float r[V];
    if (p.row_scales) {
        float m = amax[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, amax[v]);
        const float s = block_scale(slot_reduce<true>(m, warps, part[1]));
#pragma unroll
        for (int v = 0; v < V; ++v) r[v] = __frcp_rn(s);
        float *scale = p.scales + t;
        if (active && i0 == 0 && store_fits(scale, 4, p.scales, p.rows * 4, p.err)) *scale = s;
    } else {
        const int lane = threadIdx.x & 31;
        const float s = block_scale(blocks_amax<V>(amax, lane)), inv = __frcp_rn(s);
        const int v = (lane & 15) / (16 / V), k = (v * p.threads + i0) * 8 & ~127;
#pragma unroll
        for (int j = 0; j < V; ++j)
            r[j] = __shfl_sync(0xFFFFFFFFu, inv, (lane & 16) | (j * (16 / V)));
        float *scale = p.scales + t * KB + k / 128;
        if (active && lane % (16 / V) == 0 && k < p.K &&
            store_fits(scale, 4, p.scales, p.rows * KB * 4, p.err))
            *scale = s;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int k = (v * p.threads + i0) * 8;
        if (!active || k >= p.K) continue;
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 y = mul2(h[v][i], f2s(r[v]));
            c[i] = e4m3x2(f2_lo(y), f2_hi(y));
        }
        uint8_t *out = p.q + t * p.K + k;
        if (store_fits(out, 8, p.q, p.rows * p.K, p.err))
            *reinterpret_cast<uint2 *>(out) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
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

// A row's h, d_y and d_h in a thread, as they lie in memory.  With four vectors a thread
// d_h is loaded where it is used, in the registers of h, and the weight too: there is no
// room for them.
template <int DT, int V>
struct GradRow {
    static constexpr bool kLate = V == 4;
    Vec8<DT> h[V], g[V], d[kLate ? 1 : V];
    float u;
    __device__ __forceinline__ void load(const NormGradParams &p, int64_t t, int i0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int k = (v * p.threads + i0) * 8;
            h[v].zero();
            g[v].zero();
            if (!kLate) d[v].zero();
            if (k < p.K && t < p.rows) {
                h[v].load(p.h, t * p.h_stride + k);
                g[v].load(p.dy, t * p.dy_stride + k);
                if (!kLate && p.dh) d[v].load(p.dh, t * p.dh_stride + k);
            }
        }
        u = t < p.rows ? __ldg(p.rstd + t) : 0.0f;
    }
};

// AHEAD: the next row's loads are in flight while one is worked on (its registers).
template <int DT, int V, int MOST, bool AHEAD>
__global__ void __launch_bounds__(MOST) norm_grad_kernel(NormGradParams p) {
    __shared__ float part[2][32];
    pdl_wait();
    pdl_trigger();
    const int warps = p.threads >> 5, i0 = (int)threadIdx.x % p.threads;
    const int slots = blockDim.x / p.threads;
    const int64_t slot = (int64_t)blockIdx.x * slots + threadIdx.x / p.threads;
    constexpr bool kLate = GradRow<DT, V>::kLate;
    F2 dw[V][4];
    Vec8<DT> wv[kLate ? 1 : V];
    auto weight = [&](int v, F2 (&w)[4]) {
        const int k = (v * p.threads + i0) * 8;
        if (kLate) wv[0].load_kept(p.w, k < p.K ? k : 0);
        wv[kLate ? 0 : v].values(w);
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int k = (v * p.threads + i0) * 8;
        if (!kLate) wv[v % (kLate ? 1 : V)].load_kept(p.w, k < p.K ? k : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[v][i] = f2s(0.0f);
    }
    // every slot of the CTA walks the same number of rows: they share its barriers
    const int64_t step = (int64_t)gridDim.x * slots;
    const int64_t first = (int64_t)blockIdx.x * slots;
    int turn = 0;
    GradRow<DT, V> next;
    if (AHEAD) next.load(p, slot, i0);
    for (int64_t t0 = 0; first + t0 < p.rows; t0 += step, turn ^= 1) {
        const int64_t t = slot + t0;
        const bool active = t < p.rows;
        GradRow<DT, V> row;
        if (AHEAD) {
            row = next;
            next.load(p, t + step, i0);
        } else {
            row.load(p, t, i0);
        }
        F2 dot = f2s(0.0f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            F2 h[4], g[4], w[4];
            row.h[v].values(h);
            row.g[v].values(g);
            weight(v, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 gh = mul2(g[i], h[i]);
                dw[v][i] = fma2(gh, f2s(row.u), dw[v][i]);
                dot = fma2(gh, w[i], dot);
            }
        }
        const float sum =
            slot_reduce<false>(__fadd_rn(f2_lo(dot), f2_hi(dot)), warps, part[turn]);
        // d_x = u (g w - h mean(g w h) u^2) + d_h
        const F2 u = f2s(row.u);
        const F2 back = f2s(-__fmul_rn(__fdiv_rn(sum, (float)p.K), __fmul_rn(row.u, row.u)));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int k = (v * p.threads + i0) * 8;
            if (!active || k >= p.K) continue;
            F2 h[4], g[4], w[4], d[4];
            row.h[v].values(h);
            row.g[v].values(g);
            if constexpr (GradRow<DT, V>::kLate) {
                if (p.dh) row.h[v].load(p.dh, t * p.dh_stride + k);
                row.h[v].values(d);
            } else {
                row.d[v].values(d);
            }
            weight(v, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = fma2(h[i], back, mul2(g[i], w[i]));
                g[i] = p.dh ? fma2(g[i], u, d[i]) : mul2(g[i], u);
            }
            row.h[v].set(g);
            row.h[v].store(p.dx, t * p.K + k, p.rows * p.K, p.err);
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
            st_global_v4(out + 16 * i, __float_as_uint(f2_lo(dw[v][2 * i])),
                         __float_as_uint(f2_hi(dw[v][2 * i])),
                         __float_as_uint(f2_lo(dw[v][2 * i + 1])),
                         __float_as_uint(f2_hi(dw[v][2 * i + 1])));
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

Split split_into(int64_t K, int v) {
    const int vecs = (int)((K + 7) / 8);
    const int threads = ((vecs + v - 1) / v + 31) / 32 * 32;
    return {v, threads, std::max(1, 128 / threads)};
}

// As few threads as hold the row with at most four vectors each: the reduction costs each
// of them the same, and up to 1024 elements a warp has a row without a barrier.  x,
// residual to h, y, bf16, against two vectors a thread: 16384 x 7168 140 us / 165.
Split norm_split(int64_t K) { return split_into(K, K <= 256 ? 1 : K <= 512 ? 2 : 4); }

// The gradient's next row is in registers too: one vector a thread up to 256 threads, two
// up to 512, four past that (16384 x 7168 160 us with two, 314 with four).
Split grad_split(int64_t K) { return split_into(K, K <= 2048 ? 1 : K <= 16 * kMaxThreads ? 2 : 4); }

template <int DT, int V, int MOST>
cudaError_t run_norm(const NormParams &p, const Split &c, cudaStream_t s) {
    return launch_pdl(norm_kernel<DT, V, MOST>, (unsigned)((p.rows + c.slots - 1) / c.slots),
                      c.threads * c.slots, 0, s, p);
}

template <int DT>
cudaError_t run_norm_type(NormParams p, cudaStream_t s) {
    const Split c = norm_split(p.K);
    p.threads = c.threads;
    return c.v == 1             ? run_norm<DT, 1, 128>(p, c, s)
           : c.v == 2           ? run_norm<DT, 2, 128>(p, c, s)
           : c.threads <= 256   ? run_norm<DT, 4, 256>(p, c, s)
                                : run_norm<DT, 4, kMaxThreads>(p, c, s);
}

// The gradient's grid: rows of 512 to 768 threads for each of this machine's 152 SMs,
// fewer where there are fewer rows.  It depends on the sizes alone, so that the
// workspace's size does.
int grad_ctas(int64_t rows, const Split &c) {
    const int per_sm = std::max(1, (c.v == 1 ? 768 : 512) / (c.threads * c.slots));
    return (int)std::min<int64_t>((rows + c.slots - 1) / c.slots, per_sm * 152);
}

template <int DT, int V, int MOST, bool AHEAD>
cudaError_t run_grad(const NormGradParams &p, const Split &c, cudaStream_t s) {
    return launch_pdl(norm_grad_kernel<DT, V, MOST, AHEAD>, (unsigned)grad_ctas(p.rows, c),
                      c.threads * c.slots, 0, s, p);
}

template <int DT>
cudaError_t run_grad_type(NormGradParams p, cudaStream_t s) {
    const Split c = grad_split(p.K);
    p.threads = c.threads;
    return c.v == 1   ? run_grad<DT, 1, 256, true>(p, c, s)
           : c.v == 2 ? run_grad<DT, 2, kMaxThreads, DT != MOEQ_FP32>(p, c, s)
                      : run_grad<DT, 4, kMaxThreads, false>(p, c, s);
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
    const Split c = grad_split(K);
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
