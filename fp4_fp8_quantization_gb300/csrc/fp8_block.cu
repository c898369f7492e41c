// FP8 (E4M3) quantization with one fp32 scale for each block of 128: 1 x 128
// blocks of rows (activations: plain rows, tokens copied to their routed
// rows, SwiGLU of a gate/up tensor) and 128 x 128 blocks of weights.
//
//   s = max(amax / 448, 2^-126),  r = 1 / s,  q = E4M3(x * r)
//
// each step one fp32 operation, round to nearest even, saturating.  The floor
// keeps r finite; an all-zero block has the floor as its scale.  A NaN does
// not enter amax and stays a NaN code of its own element; an infinity makes
// its block's scale infinite and itself a NaN code.
//
// All are streaming kernels: 2 bytes read and 1 written per element (1 per
// choice for routed tokens, each token read and quantized once; 4 read for
// SwiGLU).  Measured, with the share of the copy rate: routed 16384 x 4096 top-8
// 102 us (0.99), rows 65536 x 4096 131 (0.92), 16384 x 7168 59 (0.89), 8192 x 4096
// 19 (0.79), weights 64 x 4096 x 7168 982 (0.85), 48 x 1880 x 2480 125 (0.79).
// SwiGLU is bound by the instructions of the SiLU, 131072 x 1536 200 (0.75), and
// below the table's sizes by having no load in flight while a warp computes:
// 8191 x 1536 16.5 (0.56).
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "tensormap.h"

namespace moeq {

namespace {

constexpr int kBlk = 128;
constexpr int kWarps = 4;

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

struct BlockParams {
    const uint16_t *in;
    int64_t stride, rows, K;
    const int32_t *dst;  // null: row t goes to row t
    int top_k;
    int64_t out_rows;
    uint8_t *out;
    float *scales;
    uint32_t *err;
};

// 8 elements of a row from 16 bytes of bf16, or, for SwiGLU, 8 values
// silu(gate) * up from 32 bytes of gate/up pairs.
template <bool SWIGLU>
struct Piece {
    uint4 u[SWIGLU ? 2 : 1];
    __device__ __forceinline__ void load(const uint16_t *row, int64_t k) {
        const uint16_t *src = row + (SWIGLU ? 2 * k : k);
        u[0] = ld_stream(src);
        if constexpr (SWIGLU) u[1] = ld_stream(src + 8);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (SWIGLU ? 2 : 1); ++i) u[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    // tab: the SiLU table, or null to compute
    __device__ __forceinline__ void values(float (&x)[8], const float *tab) const {
        if constexpr (SWIGLU) {
            const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
            for (int i = 0; i < 8; i += 2) {  // gate in the low half, up in the high
                const F2 h = tab ? swiglu2_tab(w[i], w[i + 1], tab)
                                 : swiglu2(__uint_as_float(w[i] << 16),
                                           __uint_as_float(w[i + 1] << 16),
                                           __uint_as_float(w[i] & 0xFFFF0000u),
                                           __uint_as_float(w[i + 1] & 0xFFFF0000u));
                x[i] = f2_lo(h);
                x[i + 1] = f2_hi(h);
            }
        } else {
            unpack8(u[0], x);
        }
    }
};

// U * 256 consecutive elements of a row, a warp's work: 16 lanes hold a
// block, 8 elements each.
template <bool SWIGLU, int U>
struct Item {
    Piece<SWIGLU> in[U];
    float x[U][8];
    int64_t t, k0;  // row, and the lane's first element
    // all of the loads at once
    __device__ __forceinline__ void load(const BlockParams &p, int64_t item, int segments,
                                         int lane) {
        t = item / segments;
        k0 = (item - t * segments) * (U * 256) + lane * 8;
        const uint16_t *row = p.in + t * p.stride;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (t < p.rows && k0 + i * 256 < p.K)
                in[i].load(row, k0 + i * 256);
            else
                in[i].zero();
        }
    }
    __device__ __forceinline__ void values(const float *tab) {
#pragma unroll
        for (int i = 0; i < U; ++i) in[i].values(x[i], tab);
    }
};

// Quantizes and stores the values x of the item at row t, element k0.
template <int U>
__device__ __forceinline__ void store_item(const BlockParams &p, const float (&x)[U][8], int64_t t,
                                           int64_t k0, int lane) {
    const int64_t KB = (p.K + kBlk - 1) / kBlk;
    uint2 q[U];
    float s[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        float m = amax8(x[i]);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        s[i] = block_scale(m);
        q[i] = codes8(x[i], __fdiv_rn(1.0f, s[i]));
    }
    for (int j = 0; j < (p.dst ? p.top_k : 1); ++j) {
        int64_t r = t;
        if (p.dst) {
            r = __ldg(p.dst + t * p.top_k + j);
            if (r < 0 || r >= p.out_rows) {
                if (r != -1 && k0 == 0) set_error(p.err, MOEQ_DEVERR_BAD_INDEX);
                continue;
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t k = k0 + i * 256;
            if (k >= p.K) continue;
            uint8_t *out = p.out + r * p.K + k;
            float *scale = p.scales + r * KB + k / kBlk;
            if (store_fits(out, 8, p.out, p.out_rows * p.K, p.err))
                *reinterpret_cast<uint2 *>(out) = q[i];
            if ((lane & 15) == 0 && store_fits(scale, 4, p.scales, p.out_rows * KB * 4, p.err))
                *scale = s[i];
        }
    }
}

template <bool SWIGLU, int U>
__global__ void __launch_bounds__(kWarps * 32) fp8_block_kernel(BlockParams p, int segments) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    Item<SWIGLU, U> it;
    it.load(p, (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), segments, lane);
    if (it.t >= p.rows) return;
    it.values(nullptr);
    store_item<U>(p, it.x, it.t, it.k0, lane);
}

// SwiGLU with the gates' SiLU from a table of every bf16 value (the same bits
// as computing it): persistent CTAs, each with its table.  The next item's
// loads are in flight while one is quantized.
constexpr int kTabWarps = 16, kTabCtas = 2;
template <int U>
__global__ void __launch_bounds__(kTabWarps * 32, kTabCtas)
    fp8_block_swiglu_tab_kernel(BlockParams p, int segments) {
    extern __shared__ float silu_tab[];
    build_silu_table(silu_tab);
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t items = p.rows * segments, step = (int64_t)gridDim.x * kTabWarps;
    int64_t item = (int64_t)blockIdx.x * kTabWarps + (threadIdx.x >> 5);
    Item<true, U> it;
    it.load(p, item, segments, lane);
    while (item < items) {
        it.values(silu_tab);
        const int64_t t = it.t, k0 = it.k0;
        float x[U][8];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) x[i][k] = it.x[i][k];
        item += step;
        it.load(p, item, segments, lane);
        store_item<U>(p, x, t, k0, lane);
    }
}

template <bool SWIGLU, int U>
cudaError_t run_fp8_block(const BlockParams &p, cudaStream_t s) {
    const int64_t segments = (p.K + U * 256 - 1) / (U * 256);
    const int64_t blocks = (p.rows * segments + kWarps - 1) / kWarps;
    if (blocks >= (int64_t)1 << 31) return cudaErrorNotSupported;
    return launch_pdl(fp8_block_kernel<SWIGLU, U>, (unsigned)blocks, kWarps * 32, 0, s, p,
                      (int)segments);
}

// kSiluTableBytes (32 KB) of dynamic shared memory need no opt-in.
template <int U>
cudaError_t run_swiglu_tab(const BlockParams &p, cudaStream_t s) {
    const int64_t segments = (p.K + U * 256 - 1) / (U * 256);
    const int64_t blocks = (p.rows * segments + kTabWarps - 1) / kTabWarps;
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, sm_count() * kTabCtas);
    return launch_pdl(fp8_block_swiglu_tab_kernel<U>, grid, kTabWarps * 32, kSiluTableBytes, s, p,
                      (int)segments);
}

// One CTA per 128 x 128 weight block (grid: K blocks, N blocks, experts): 16
// threads hold a row's 128 columns, 16 rows at a time.
__global__ void __launch_bounds__(256) fp8_block_weight_kernel(const uint16_t *w, int64_t N,
                                                               int64_t K, uint8_t *out,
                                                               float *scales, uint32_t *err) {
    pdl_wait();
    pdl_trigger();
    __shared__ float part[8];
    const int64_t e = blockIdx.z, n0 = (int64_t)blockIdx.y * kBlk;
    const int64_t k = (int64_t)blockIdx.x * kBlk + (threadIdx.x & 15) * 8;
    uint4 u[8];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t n = n0 + i * 16 + (threadIdx.x >> 4);
        u[i] = make_uint4(0u, 0u, 0u, 0u);
        if (n < N && k < K) u[i] = *reinterpret_cast<const uint4 *>(w + (e * N + n) * K + k);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x[8];
        unpack8(u[i], x);
        m = fmaxf(m, amax8(x));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, part[i]);
    const float s = block_scale(m), r = __fdiv_rn(1.0f, s);
    float *scale = scales + (e * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
    if (threadIdx.x == 0 &&
        store_fits(scale, 4, scales, (int64_t)gridDim.z * gridDim.y * gridDim.x * 4, err))
        *scale = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t n = n0 + i * 16 + (threadIdx.x >> 4);
        float x[8];
        unpack8(u[i], x);
        uint8_t *o = out + (e * N + n) * K + k;
        if (n < N && k < K && store_fits(o, 8, out, (int64_t)gridDim.z * N * K, err))
            *reinterpret_cast<uint2 *>(o) = codes8(x, r);
    }
}

}  // namespace

cudaError_t launch_fp8_block(const Fp8BlockArgs &a, cudaStream_t s) {
    const BlockParams p{static_cast<const uint16_t *>(a.in), a.stride, a.rows, a.K, a.dst,
                        a.top_k, a.out_rows, a.out, a.scales, a.err};
    // of at most 4 (3 with SwiGLU) loads per lane the most that leave the fewest
    // of a row's last warp without an element: 13119 x 592 SwiGLU 19.1 us with 2
    // of them, 14.7 with 3; 5775 x 1376 rows 8.7 us with 4, 6.7 with 3
    const int64_t n = (a.K + 255) / 256;
    int u = 1;
    for (int i = 2; i <= (a.swiglu ? 3 : 4); ++i)
        if ((n + i - 1) / i * i <= (n + u - 1) / u * u) u = i;
    if (!a.swiglu)
        return u == 1   ? run_fp8_block<false, 1>(p, s)
               : u == 2 ? run_fp8_block<false, 2>(p, s)
               : u == 3 ? run_fp8_block<false, 3>(p, s)
                        : run_fp8_block<false, 4>(p, s);
    // the table pays for its construction from about 2^25 values on: 8191 x 1536
    // 16.5 us computed, 19.1 by table; 32768 x 1536 57.9 and 53.7; 131072 x 1536
    // 222 and 200
    if (a.rows * a.K < (int64_t)1 << 25)
        return u == 1   ? run_fp8_block<true, 1>(p, s)
               : u == 2 ? run_fp8_block<true, 2>(p, s)
                        : run_fp8_block<true, 3>(p, s);
    return u == 1   ? run_swiglu_tab<1>(p, s)
           : u == 2 ? run_swiglu_tab<2>(p, s)
                    : run_swiglu_tab<3>(p, s);
}

cudaError_t launch_fp8_block_weight(const void *w, int64_t E, int64_t N, int64_t K, uint8_t *out,
                                    float *scales, uint32_t *err, cudaStream_t s) {
    const dim3 grid((unsigned)((K + kBlk - 1) / kBlk), (unsigned)((N + kBlk - 1) / kBlk), (unsigned)E);
    return launch_pdl(fp8_block_weight_kernel, grid, 256, 0, s, static_cast<const uint16_t *>(w), N,
                      K, out, scales, err);
}

}  // namespace moeq
