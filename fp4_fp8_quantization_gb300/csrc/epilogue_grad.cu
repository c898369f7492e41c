// Gradient of the block product's epilogue c = act(z) + residual, z = product +
// bias[e], over ragged groups:
//
//   d_z = d_c act'(z)   as E4M3 codes with a scale for each 1 x 128 block, ready for
//                       the product with the transposed weights, and / or as bf16
//   d_bias[e] = sum over the rows of expert e of d_z (fp32, before any rounding)
//
// One pass: 4 bytes read and 1 (or 3) written per element.  A CTA takes tiles of
// 64 to 512 rows of one group by 256 columns, a warp a row at a time, 16 lanes a
// block; each thread sums its 8 columns over its rows, the warps join in shared
// memory, and a tile leaves one row of partial sums.  A second kernel adds an
// expert's rows of them in the order of groups and tiles: no atomics, the same
// bits every time.  Four rows of a warp are worked on together, so that their 8 block
// scales take one division a lane, and the next four's loads are in flight meanwhile.
//
// 32768 x 4096 over 64 experts, silu, even groups: 127 us (0.78 of the copy rate,
// of it 6 for the bias's second kernel), 0.59 of DRAM's peak and 0.65 of the issue slots
// in the profile: instructions and the tiles' beginnings, which nothing overlaps.  4096 x
// 4096 23, 64 x 4096 7.4 (4.9 without the bias).
#include <algorithm>

#include "activation.cuh"
#include "common.cuh"
#include "fp8_block.cuh"
#include "launch.h"
#include "tensormap.h"

namespace moeq {

namespace {

constexpr int kWarps = 8;
constexpr int kCols = 256;  // of a CTA: 32 lanes of 8

__device__ __forceinline__ void pairs8(const uint4 &u, F2 (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

struct EpilogueGradParams {
    const uint16_t *dc, *z;
    int64_t dc_stride, rows, N;
    int tile_rows;
    const uint32_t *offsets;
    const int32_t *expert_ids;
    int num_groups, num_experts;
    uint8_t *q;
    float *scales;
    uint16_t *dz;
    float *part;       // [tiles][N], or null
    uint32_t *tiles;   // [groups + 1] tiles before each group, with part
    int64_t max_tiles;
    uint32_t *err;
};

// The largest of 4 rows' m over the 16 lanes of a block: lane l of them gets that of
// row l / 4 (each step sends the rows that the other half of the lanes keeps).
__device__ __forceinline__ float rows_amax(const float (&m)[4], int lane) {
    constexpr unsigned kAll = 0xFFFFFFFFu;
    const bool b3 = lane & 8, b2 = lane & 4;
    const float k0 = fmaxf(b3 ? m[2] : m[0], __shfl_xor_sync(kAll, b3 ? m[0] : m[2], 8));
    const float k1 = fmaxf(b3 ? m[3] : m[1], __shfl_xor_sync(kAll, b3 ? m[1] : m[3], 8));
    float k = fmaxf(b2 ? k1 : k0, __shfl_xor_sync(kAll, b2 ? k0 : k1, 4));
    k = fmaxf(k, __shfl_xor_sync(kAll, k, 2));
    return fmaxf(k, __shfl_xor_sync(kAll, k, 1));
}

template <int ACT>
__global__ void __launch_bounds__(kWarps * 32, 2) epilogue_grad_kernel(EpilogueGradParams p) {
    // tiles before each group
    __shared__ uint32_t prefix[kMaxGroups + 1];
    __shared__ float sums[kWarps][kCols];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = p.num_groups;
    const bool first = blockIdx.x == 0 && blockIdx.y == 0;
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
        const uint32_t r0 = __ldg(p.offsets + g), r1 = __ldg(p.offsets + g + 1);
        const int e = __ldg(p.expert_ids + g);
        uint32_t n = 0;
        if (r1 < r0 || (int64_t)r1 > p.rows) {
            if (first) set_error(p.err, MOEQ_DEVERR_BAD_OFFSETS);
        } else if (e < 0 || e >= p.num_experts) {
            if (first) set_error(p.err, MOEQ_DEVERR_BAD_EXPERT);
        } else {
            n = (r1 - r0 + p.tile_rows - 1) / p.tile_rows;
        }
        prefix[g + 1] = n;
    }
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    if (warp == 0) {  // inclusive prefix over prefix[1 .. G]
        uint32_t carry = 0;
        for (int base = 0; base < G; base += 32) {
            const int g = base + lane;
            uint32_t v = g < G ? prefix[g + 1] : 0u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o) v += t;
            }
            if (g < G) prefix[g + 1] = carry + v;
            carry += __shfl_sync(0xFFFFFFFFu, v, 31);
        }
    }
    __syncthreads();
    if (first && p.part)
        for (int g = threadIdx.x; g <= G; g += blockDim.x) {
            uint32_t *o = p.tiles + g;
            if (store_fits(o, 4, p.tiles, (int64_t)(G + 1) * 4, p.err)) *o = prefix[g];
        }
    // groups that overlap can have more tiles than the workspace has rows
    uint32_t total = prefix[G];
    if ((int64_t)total > p.max_tiles) {
        if (first && threadIdx.x == 0) set_error(p.err, MOEQ_DEVERR_BAD_OFFSETS);
        total = (uint32_t)p.max_tiles;
    }
    const int64_t n = (int64_t)blockIdx.x * kCols + lane * 8, NB = (p.N + 127) / 128;
    const bool in_n = n < p.N;
    for (uint32_t t = blockIdx.y; t < total; t += gridDim.y) {
        int lo = 0, hi = G;  // the last group that begins at or before tile t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= t) lo = mid; else hi = mid;
        }
        const int64_t r0 = (int64_t)__ldg(p.offsets + lo) + (int64_t)(t - prefix[lo]) * p.tile_rows;
        const int rows = (int)min((int64_t)p.tile_rows, (int64_t)__ldg(p.offsets + lo + 1) - r0);
        F2 sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = f2s(0.0f);
        constexpr int U = 4;  // rows of a warp that are worked on together
        uint4 dc[U], zv[U];
        auto load = [&](int base) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t r = r0 + base + j * kWarps;
                dc[j] = zv[j] = make_uint4(0u, 0u, 0u, 0u);
                if (base + j * kWarps < rows && in_n) {
                    dc[j] = ld_stream(p.dc + r * p.dc_stride + n);
                    if (ACT != MOEQ_ACT_NONE) zv[j] = ld_stream(p.z + r * p.N + n);
                }
            }
        };
        load(warp);
        for (int base = warp; base < rows; base += U * kWarps) {
            F2 x[U][4];
            float m[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                pairs8(dc[j], x[j]);
                if constexpr (ACT != MOEQ_ACT_NONE) {
                    F2 z[4];
                    pairs8(zv[j], z);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[j][i] = mul2(x[j][i], slope2<ACT>(z[i]));
                }
                m[j] = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[i] = add2(sum[i], x[j][i]);
                    m[j] = fmaxf(fmaxf(m[j], fabsf(f2_lo(x[j][i]))), fabsf(f2_hi(x[j][i])));
                }
            }
            load(base + U * kWarps);  // on their way while these are quantized and stored
            float inv = 0.0f;  // of row (lane / 4) % 4
            if (p.q) {
                const float s = block_scale(rows_amax(m, lane));
                inv = __frcp_rn(s);
                const int j = (lane >> 2) & 3;
                const int64_t r = r0 + base + j * kWarps;
                // 128-column blocks: the lanes 0 and 16 begin one
                const int64_t at = (int64_t)blockIdx.x * (kCols / 128) + (lane >> 4);
                float *scale = p.scales + r * NB + at;
                if ((lane & 3) == 0 && base + j * kWarps < rows && at < NB &&
                    store_fits(scale, 4, p.scales, p.rows * NB * 4, p.err))
                    *scale = s;
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t r = r0 + base + j * kWarps;
                const float rj = __shfl_sync(0xFFFFFFFFu, inv, (lane & 16) | (j << 2));
                if (base + j * kWarps >= rows || !in_n) continue;
                if (p.q) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 y = mul2(x[j][i], f2s(rj));
                        w[i] = e4m3x2(f2_lo(y), f2_hi(y));
                    }
                    uint8_t *out = p.q + r * p.N + n;
                    if (store_fits(out, 8, p.q, p.rows * p.N, p.err))
                        *reinterpret_cast<uint2 *>(out) =
                            make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
                }
                if (p.dz) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = f32_to_bf16_bits(f2_lo(x[j][i])) |
                               (f32_to_bf16_bits(f2_hi(x[j][i])) << 16);
                    uint16_t *out = p.dz + r * p.N + n;
                    if (store_fits(out, 16, p.dz, p.rows * p.N * 2, p.err))
                        st_global_v4(out, w[0], w[1], w[2], w[3]);
                }
            }
        }
        if (!p.part) continue;
        __syncthreads();  // the sums of the tile before have been read
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sums[warp][lane * 8 + 2 * i] = f2_lo(sum[i]);
            sums[warp][lane * 8 + 2 * i + 1] = f2_hi(sum[i]);
        }
        __syncthreads();
        const int64_t col = (int64_t)blockIdx.x * kCols + threadIdx.x;
        float v = sums[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = __fadd_rn(v, sums[w][threadIdx.x]);
        float *out = p.part + (int64_t)t * p.N + col;
        if (col < p.N && store_fits(out, 4, p.part, p.max_tiles * p.N * 4, p.err)) *out = v;
    }
}

// d_bias[e] from the tiles' sums: 128 columns a CTA, its warps take an expert's tiles
// in turn and join.
__global__ void __launch_bounds__(1024) bias_grad_kernel(const float *part, const uint32_t *tiles,
                                                         int64_t max_tiles,
                                                         const int32_t *expert_ids, int G,
                                                         int64_t N, float *d_bias, int E,
                                                         uint32_t *err) {
    __shared__ float4 sums[32][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t n = (int64_t)blockIdx.x * 128 + lane * 4;  // N is a multiple of 8
    const int e = blockIdx.y;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](const float4 &u) {
        v.x = __fadd_rn(v.x, u.x);
        v.y = __fadd_rn(v.y, u.y);
        v.z = __fadd_rn(v.z, u.z);
        v.w = __fadd_rn(v.w, u.w);
    };
    for (int base = 0; base < G; base += 32) {
        const int g = base + lane;
        uint32_t mine = __ballot_sync(0xFFFFFFFFu, g < G && __ldg(expert_ids + g) == e);
        for (; mine; mine &= mine - 1) {
            const int at = base + __ffs((int)mine) - 1;
            const int64_t t1 = min((int64_t)__ldg(tiles + at + 1), max_tiles);
            if (n < N) {
#pragma unroll 4
                for (int64_t t = (int64_t)__ldg(tiles + at) + warp; t < t1; t += warps)
                    add(__ldg(reinterpret_cast<const float4 *>(part + t * N + n)));
            }
        }
    }
    sums[warp][lane] = v;
    __syncthreads();
    if (warp == 0) {
        for (int w = 1; w < warps; ++w) add(sums[w][lane]);
        float *out = d_bias + (int64_t)e * N + n;
        if (n < N && store_fits(out, 16, d_bias, (int64_t)E * N * 4, err))
            st_global_v4(out, __float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                         __float_as_uint(v.w));
    }
}

}  // namespace

cudaError_t launch_epilogue_grad(const EpilogueGradArgs &a, cudaStream_t s) {
    const int64_t tiles = epilogue_grad_tiles(a.groups.total_rows, a.N, a.groups.num_groups);
    // its parts: the table of tiles, then the sums, 16-byte aligned
    uint32_t *table = static_cast<uint32_t *>(a.workspace);
    float *part = a.d_bias ? reinterpret_cast<float *>(
                                 static_cast<uint8_t *>(a.workspace) +
                                 epilogue_grad_table_bytes(a.groups.num_groups))
                           : nullptr;
    const EpilogueGradParams p{static_cast<const uint16_t *>(a.dc),
                               static_cast<const uint16_t *>(a.z), a.dc_stride,
                               a.groups.total_rows, a.N,
                               (int)epilogue_grad_rows(a.groups.total_rows, a.N),
                               a.groups.row_offsets,
                               a.groups.expert_ids, a.groups.num_groups, a.groups.num_experts, a.q,
                               a.scales, static_cast<uint16_t *>(a.dz), part, table, tiles, a.err};
    if (tiles > 0) {
        const dim3 grid((unsigned)((a.N + kCols - 1) / kCols),
                        (unsigned)std::min<int64_t>(tiles, 65535));
        auto *kern = a.act == MOEQ_ACT_RELU   ? epilogue_grad_kernel<MOEQ_ACT_RELU>
                     : a.act == MOEQ_ACT_SILU ? epilogue_grad_kernel<MOEQ_ACT_SILU>
                     : a.act == MOEQ_ACT_GELU ? epilogue_grad_kernel<MOEQ_ACT_GELU>
                     : a.act == MOEQ_ACT_GELU_TANH
                         ? epilogue_grad_kernel<MOEQ_ACT_GELU_TANH>
                         : epilogue_grad_kernel<MOEQ_ACT_NONE>;
        const cudaError_t e = launch_pdl(kern, grid, kWarps * 32, 0, s, p);
        if (e != cudaSuccess) return e;
    }
    if (!a.d_bias) return cudaSuccess;
    // many warps where there are few CTAs
    const int64_t cols = (a.N + 127) / 128, ctas = cols * a.groups.num_experts;
    const unsigned threads = ctas < 2 * sm_count() ? 1024 : 128;
    return launch_pdl(bias_grad_kernel, dim3((unsigned)cols, (unsigned)a.groups.num_experts),
                      threads, 0, s, (const float *)part, (const uint32_t *)table, tiles,
                      a.groups.expert_ids, tiles > 0 ? a.groups.num_groups : 0, a.N, a.d_bias,
                      a.groups.num_experts, a.err);
}

}  // namespace moeq
