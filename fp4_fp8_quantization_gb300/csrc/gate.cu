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
// one pass over memory each way.  Lane l holds logits l NV .. l NV + NV - 1,
// read as vectors, so that among equal logits the lowest lane has the lowest
// index.  Selection compares order-preserving integer images of the logits;
// each lane keeps its best one at hand, and a round is one warp maximum of
// those.  16-bit logits carry their index in the low half of the image, which
// makes every image distinct.  Sums are fp32 in a fixed order.
#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.h"

namespace moeq {

namespace {

constexpr uint32_t kNegInfKey = 0x007FFFFFu;  // order_key(-inf)
constexpr int kGateWarps = 4;

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

// The same of a 16-bit logit, in 16 bits.
template <int DT>
__device__ __forceinline__ uint32_t order_key16(float x) {
    const uint32_t b = bits_of<DT>(__fadd_rn(x, 0.0f));  // exact: x came from 16 bits
    if (x != x) return 0u;
    return b ^ ((b >> 15) ? 0xFFFFu : 0x8000u);
}

template <int DT>
__device__ __forceinline__ float key16_value(uint32_t k) {
    return logit_of<DT>(k ^ ((k >> 15) ? 0x8000u : 0xFFFFu));
}

// order_key16(-inf)
template <int DT>
constexpr uint32_t kNegInfKey16 = DT == MOEQ_BF16 ? 0x007Fu : 0x03FFu;

// exp(x - m) for x <= m: within 2 + 1.2 |x - m| ulp, NaN for a NaN or for
// infinity minus infinity.
__device__ __forceinline__ float exp_diff(float x, float m) { return __expf(__fadd_rn(x, -m)); }

// Sum over groups of LANES consecutive lanes, the same in each of them.
template <int LANES = 32>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
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

template <int DT, int NV>
__device__ __forceinline__ void store_row(uint8_t *row, int E, int j0, bool vec,
                                          const float (&g)[NV]) {
    constexpr int kBytes = NV * kSize<DT>;
    if (vec && j0 + NV <= E && kBytes >= 8) {
        uint8_t *a = row + (int64_t)j0 * kSize<DT>;
        uint32_t w[kBytes < 8 ? 2 : kBytes / 4];
#pragma unroll
        for (int i = 0; i < (kBytes < 8 ? 0 : kBytes / 4); ++i)
            w[i] = DT == MOEQ_FP32
                       ? bits_of<DT>(g[i % NV])
                       : bits_of<DT>(g[2 * i % NV]) | (bits_of<DT>(g[(2 * i + 1) % NV]) << 16);
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                st_global_v4(a + 16 * i, w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
            *reinterpret_cast<uint2 *>(a) = make_uint2(w[0], w[1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (j0 + i < E) store_logit<DT>(row, j0 + i, g[i]);
    }
}

// A lane's candidates; take(own) removes the best one in the lane where own.
//
// fp32, up to 8: images and indices, sorted (an odd-even transposition sort,
// which keeps equal ones in the order of their indices).
template <int DT, int NV>
struct Candidates {
    uint32_t key[NV];
    int idx[NV];
    __device__ __forceinline__ uint32_t best() const { return key[0]; }
    __device__ __forceinline__ int at() const { return idx[0]; }
    __device__ __forceinline__ void init(const float (&x)[NV], int) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            key[i] = order_key(x[i]);
            idx[i] = i;
        }
#pragma unroll
        for (int pass = 0; pass < NV; ++pass)
#pragma unroll
            for (int i = pass & 1; i + 1 < NV; i += 2) {
                const bool swap = key[i + 1] > key[i];
                const uint32_t k = max(key[i], key[i + 1]);
                key[i + 1] = min(key[i], key[i + 1]);
                key[i] = k;
                const int a = swap ? idx[i + 1] : idx[i];
                idx[i + 1] = swap ? idx[i] : idx[i + 1];
                idx[i] = a;
            }
    }
    __device__ __forceinline__ void take(bool own) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            key[i] = own ? (i + 1 < NV ? key[(i + 1) % NV] : 0u) : key[i];
            if (i + 1 < NV) idx[i] = own ? idx[(i + 1) % NV] : idx[i];
        }
    }
};

// fp32, more: images in index order; the best is found again by a scan.
template <int NV>
struct ScannedCandidates {
    uint32_t key[NV];
    uint32_t top;
    int pos;
    __device__ __forceinline__ uint32_t best() const { return top; }
    __device__ __forceinline__ int at() const { return pos; }
    __device__ __forceinline__ void init(const float (&x)[NV], int) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = order_key(x[i]);
        scan();
    }
    __device__ __forceinline__ void scan() {
        top = 0u;
        pos = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] > top) {  // the lowest index of equal ones
                top = key[i];
                pos = i;
            }
    }
    __device__ __forceinline__ void take(bool own) {
        if (!own) return;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i == pos) key[i] = 0u;
        scan();
    }
};
template <>
struct Candidates<MOEQ_FP32, 16> : ScannedCandidates<16> {};
template <>
struct Candidates<MOEQ_FP32, 32> : ScannedCandidates<32> {};

// 16-bit logits: images that hold the index, sorted; the best is the first.
template <int DT, int NV>
struct SortedCandidates {
    uint32_t key[NV];
    __device__ __forceinline__ uint32_t best() const { return key[0]; }
    __device__ __forceinline__ void init(const float (&x)[NV], int j0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            key[i] = (order_key16<DT>(x[i]) << 16) | (uint32_t)(0xFFFF - (j0 + i));
        // odd-even merge sort, largest first (NV is a power of two)
#pragma unroll
        for (int n = 1; n < NV; n *= 2)
#pragma unroll
            for (int h = n; h >= 1; h /= 2)
#pragma unroll
                for (int a = h % n; a + h < NV; a += 2 * h)
#pragma unroll
                    for (int b = 0; b < h; ++b)
                        if (a + b + h < NV && (a + b) / (2 * n) == (a + b + h) / (2 * n)) {
                            const uint32_t u = key[a + b], v = key[a + b + h];
                            key[a + b] = max(u, v);
                            key[a + b + h] = min(u, v);
                        }
    }
    __device__ __forceinline__ void take(bool own) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            key[i] = own ? (i + 1 < NV ? key[(i + 1) % NV] : 0u) : key[i];
    }
};
template <int NV>
struct Candidates<MOEQ_BF16, NV> : SortedCandidates<MOEQ_BF16, NV> {};
template <int NV>
struct Candidates<MOEQ_FP16, NV> : SortedCandidates<MOEQ_FP16, NV> {};

template <int DT, int NV>
__global__ void __launch_bounds__(kGateWarps * 32) gate_kernel(GateParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5);
    if (t >= p.num_tokens) return;
    float x[NV];
    load_row<DT>(p.logits + t * p.stride, p.E, lane * NV, rows_aligned<DT, NV>(p.stride), x);
    Candidates<DT, NV> c;
    c.init(x, lane * NV);
    // lane r: choice r.  A round past the last logit above -inf finds an image
    // that is not above kNegInf and is dropped below.
    int my_j = 0;
    uint32_t my_key = 0u, top = 0u;
    for (int r = 0; r < p.top_k; ++r) {
        const uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, c.best());
        int j = 0;
        if constexpr (DT == MOEQ_FP32) {
            const int owner = __ffs((int)__ballot_sync(0xFFFFFFFFu, c.best() == mx)) - 1;
            j = owner * NV + __shfl_sync(0xFFFFFFFFu, c.at(), owner);
            c.take(lane == owner);
        } else {
            c.take(c.best() == mx);  // images are distinct
        }
        if (r == 0) top = mx;
        if (lane == r) {
            my_j = j;
            my_key = mx;
        }
    }
    constexpr uint32_t kNone = DT == MOEQ_FP32 ? kNegInfKey : (kNegInfKey16<DT> << 16 | 0xFFFFu);
    int id = -1;
    float w = 0.0f;
    if (top > kNone) {
        float m, e = 0.0f;
        if constexpr (DT == MOEQ_FP32) {
            m = key_value(top);
            if (my_key > kNone) {
                id = my_j;
                e = exp_diff(key_value(my_key), m);
            }
        } else {
            m = key16_value<DT>(top >> 16);
            if (my_key > kNone) {
                id = 0xFFFF - (int)(my_key & 0xFFFFu);
                e = exp_diff(key16_value<DT>(my_key >> 16), m);
            }
        }
        // a NaN logit, or m infinite, makes either denominator NaN
        float total = 0.0f;
        if (p.normalize) {
            bool nan = false;
#pragma unroll
            for (int i = 0; i < NV; ++i) nan |= x[i] != x[i];
            total = lanes_sum(e);
            if (__any_sync(0xFFFFFFFFu, nan)) total = __int_as_float(0x7FFFFFFF);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) total = __fadd_rn(total, exp_diff(x[i], m));
            total = lanes_sum(total);
        }
        w = __fmul_rn(__fdiv_rn(e, total), p.scale);
    }
    if (lane < p.top_k && store_ok(t < p.num_tokens, p.err)) {
        p.ids[t * p.top_k + lane] = id;
        p.weights[t * p.top_k + lane] = w;
    }
}

// Many tokens, few experts, top_k <= KC: a lane per token.  A warp brings 32
// columns of its 32 tokens through shared memory (whole lines in, a column out
// per lane, rows 33 words apart so that neither side has bank conflicts), and
// each lane keeps the sorted list of its best KC, entering a logit only above
// the last of them, so that among equal ones the lowest index stays first.
// The sum of the plain weights runs along with the list's first as maximum.
template <int DT, int KC>
__global__ void __launch_bounds__(kGateWarps * 32) gate_rows_kernel(GateParams p) {
    __shared__ float tiles[kGateWarps][32 * 33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    float *tile = tiles[threadIdx.x >> 5];
    const int64_t t0 = ((int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5)) * 32;
    if (t0 >= p.num_tokens) return;
    const int rows = (int)(p.num_tokens - t0 < 32 ? p.num_tokens - t0 : 32);
    const uint8_t *in = p.logits + t0 * p.stride;
    float v[KC], total = 0.0f;
    int id[KC];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        v[i] = -kInf;
        id[i] = -1;
    }
    for (int c0 = 0; c0 < p.E; c0 += 32) {
        const int cols = min(p.E - c0, 32);
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 8) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = r0 + i < rows && lane < cols
                           ? load_logit<DT>(in + (r0 + i) * p.stride, c0 + lane)
                           : -kInf;
#pragma unroll
            for (int i = 0; i < 8; ++i) tile[(r0 + i) * 33 + lane] = x[i];
        }
        __syncwarp();
        const float m0 = v[0];
#pragma unroll 4
        for (int c = 0; c < cols; ++c) {
            const float x = tile[lane * 33 + c];
            nan |= x != x;
            if (x > v[KC - 1]) {
                v[KC - 1] = x;
                id[KC - 1] = c0 + c;
#pragma unroll
                for (int i = KC - 1; i > 0; --i) {
                    const bool up = v[i] > v[i - 1];
                    const float a = v[i - 1], b = v[i];
                    const int ia = id[i - 1], ib = id[i];
                    v[i - 1] = up ? b : a;
                    v[i] = up ? a : b;
                    id[i - 1] = up ? ib : ia;
                    id[i] = up ? ia : ib;
                }
            }
        }
        if (!p.normalize && v[0] > -kInf) {
            float part = 0.0f;
#pragma unroll 4
            for (int c = 0; c < cols; ++c)
                part = __fadd_rn(part, exp_diff(tile[lane * 33 + c], v[0]));
            total = __fmaf_rn(total, exp_diff(m0, v[0]), part);
        }
        __syncwarp();
    }
    float e[KC], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        e[i] = i < p.top_k && id[i] >= 0 ? exp_diff(v[i], v[0]) : 0.0f;
        sum = __fadd_rn(sum, e[i]);
    }
    if (p.normalize) total = sum;
    if (nan) total = __int_as_float(0x7FFFFFFF);
    // ids and weights leave through shared memory, in whole lines
    float *ids = tile, *w = tile + 32 * KC;
#pragma unroll
    for (int i = 0; i < KC; ++i)
        if (i < p.top_k) {
            ids[lane * p.top_k + i] = __int_as_float(id[i]);
            w[lane * p.top_k + i] =
                id[0] < 0 ? 0.0f : __fmul_rn(__fdiv_rn(e[i], total), p.scale);
        }
    __syncwarp();
    const int64_t at = t0 * p.top_k;
    for (int i = lane; i < rows * p.top_k; i += 32)
        if (store_ok(at + i < p.num_tokens * p.top_k, p.err)) {
            p.ids[at + i] = __float_as_int(ids[i]);
            p.weights[at + i] = w[i];
        }
}

// The gradient: LANES lanes per token (top_k <= LANES), each with V vectors of
// 16 bytes of the row (coalesced), so that the sums over lanes are shared by
// the 32 / LANES tokens of a warp.  Every logit's part of the row is stored
// first, then the chosen ones over it.
template <int DT, int LANES, int V>
__global__ void __launch_bounds__(kGateWarps * 32) gate_grad_kernel(GateParams p, int vec) {
    pdl_wait();
    pdl_trigger();
    constexpr int W = 16 / kSize<DT>;  // logits per vector
    const int lane = threadIdx.x & 31, sub = lane % LANES;
    const int64_t slot = ((int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5)) * (32 / LANES) +
                         lane / LANES;
    const bool active = slot < p.num_tokens;
    const int64_t t = active ? slot : p.num_tokens - 1;
    const uint8_t *in = p.logits + t * p.stride;
    float x[V][W];
#pragma unroll
    for (int i = 0; i < V; ++i) load_row<DT>(in, p.E, (i * LANES + sub) * W, vec & 1, x[i]);
    int id = -1;
    float d = 0.0f, e = 0.0f;  // lane r: s d_w_r and exp(x_{i_r} - m) of choice r
    if (sub < p.top_k) {
        id = __ldg(p.ids + t * p.top_k + sub);
        if (id < -1 || id >= p.E) {
            if (active) set_error(p.err, MOEQ_DEVERR_BAD_EXPERT);
            id = -1;
        }
        if (id >= 0) d = __fmul_rn(__ldg(p.d_weights + t * p.top_k + sub), p.scale);
    }
    const float chosen = id >= 0 ? load_logit<DT>(in, id) : 0.0f;
    float m = -kInf;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < W; ++k) {
            m = fmaxf(m, x[i][k]);
            nan |= x[i][k] != x[i][k];
        }
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const bool some = m > -kInf;
    if (id >= 0 && some) e = exp_diff(chosen, m);
    float total = nan ? __int_as_float(0x7FFFFFFF) : e;
    if (!p.normalize) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < W; ++k) {
                x[i][k] = some ? exp_diff(x[i][k], m) : 0.0f;
                total = __fadd_rn(total, x[i][k]);
            }
    }
    total = lanes_sum<LANES>(total);
    const float inv = some ? __fdiv_rn(1.0f, total) : 0.0f;
    const float q = __fmul_rn(e, inv);
    const float mean = lanes_sum<LANES>(id >= 0 ? __fmul_rn(q, d) : 0.0f);
    const float part = __fmul_rn(-mean, inv);
    constexpr int64_t kS = kSize<DT>;
    uint8_t *out = p.d_logits + t * p.E * kS;
    if (active && store_ok(t < p.num_tokens, p.err)) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float g[W];
#pragma unroll
            for (int k = 0; k < W; ++k) g[k] = p.normalize ? 0.0f : __fmul_rn(part, x[i][k]);
            store_row<DT>(out, p.E, (i * LANES + sub) * W, vec & 2, g);
        }
    }
    __syncwarp();  // orders the stores above before those below
    if (active && id >= 0) store_logit<DT>(out, id, __fmul_rn(q, __fadd_rn(d, -mean)));
}

template <int DT>
cudaError_t run_grad(const GateParams &p, cudaStream_t s) {
    constexpr int kS = kSize<DT>;
    const int vec = (p.stride % 16 == 0) | (p.E * kS % 16 == 0 ? 2 : 0);
    const int per8 = 8 * 16 / kS;  // logits of 8 lanes with one vector each
    const int nv = (p.E + per8 - 1) / per8;
    auto go = [&](void (*kern)(GateParams, int), int lanes) {
        const int64_t per_cta = kGateWarps * 32 / lanes;
        return launch_pdl(kern, (unsigned)((p.num_tokens + per_cta - 1) / per_cta), kGateWarps * 32,
                          0, s, p, vec);
    };
    if (p.top_k <= 8 && nv <= 1) return go(gate_grad_kernel<DT, 8, 1>, 8);
    if (p.top_k <= 8 && nv <= 2) return go(gate_grad_kernel<DT, 8, 2>, 8);
    if (p.top_k <= 8 && nv <= 4) return go(gate_grad_kernel<DT, 8, 4>, 8);
    if (nv <= 4) return go(gate_grad_kernel<DT, 32, 1>, 32);
    if (nv <= 8) return go(gate_grad_kernel<DT, 32, 2>, 32);
    if (nv <= 16) return go(gate_grad_kernel<DT, 32, 4>, 32);
    return go(gate_grad_kernel<DT, 32, 8>, 32);
}

template <int DT>
cudaError_t run_gate(const GateParams &p, cudaStream_t s) {
    // a lane per token once that fills the GPU and the rows are short: 131072 x
    // 32, top-8 15.0 us against 34.6 with a warp per token, 32768 x 64 11.2
    // against 11.1, 8192 x 64 9.5 against 4.3, 65537 x 128 34.4 against 28.8
    if (p.top_k <= 8 && p.E <= 64 && p.num_tokens >= 1024 * (int64_t)p.E)
        return launch_pdl(p.top_k <= 2   ? gate_rows_kernel<DT, 2>
                          : p.top_k <= 4 ? gate_rows_kernel<DT, 4>
                                         : gate_rows_kernel<DT, 8>,
                          (unsigned)((p.num_tokens + 32 * kGateWarps - 1) / (32 * kGateWarps)),
                          kGateWarps * 32, 0, s, p);
    const unsigned blocks = (unsigned)((p.num_tokens + kGateWarps - 1) / kGateWarps);
    const int nv = (p.E + 31) / 32;
    void (*kern)(GateParams) = nv <= 1    ? gate_kernel<DT, 1>
                               : nv <= 2  ? gate_kernel<DT, 2>
                               : nv <= 4  ? gate_kernel<DT, 4>
                               : nv <= 8  ? gate_kernel<DT, 8>
                               : nv <= 16 ? gate_kernel<DT, 16>
                                          : gate_kernel<DT, 32>;
    return launch_pdl(kern, blocks, kGateWarps * 32, 0, s, p);
}

template <int DT>
cudaError_t run(const GateParams &p, cudaStream_t s) {
    return p.d_logits ? run_grad<DT>(p, s) : run_gate<DT>(p, s);
}

}  // namespace

cudaError_t launch_gate(const GateArgs &a, cudaStream_t s) {
    const int64_t size = a.dtype == MOEQ_FP32 ? 4 : 2;
    GateParams p{static_cast<const uint8_t *>(a.logits), a.stride * size, a.num_tokens,
                 a.num_experts, a.top_k, a.normalize, a.scale, a.ids, a.weights, a.d_weights,
                 static_cast<uint8_t *>(a.d_logits), a.err};
    if (a.dtype == MOEQ_BF16) return run<MOEQ_BF16>(p, s);
    if (a.dtype == MOEQ_FP16) return run<MOEQ_FP16>(p, s);
    return run<MOEQ_FP32>(p, s);
}

}  // namespace moeq
