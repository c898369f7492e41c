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
// The whole row of a token is in the registers of L lanes (32, or 8 or 16 of a
// warp where there are many tokens; E <= 1024), one pass over memory each way.
// Lane l of them holds logits l NV .. l NV + NV - 1, read as vectors, so that
// among equal logits the lowest lane has the lowest index.  Selection compares
// order-preserving integer images of the logits that hold the index in their
// low bits, so that a round is one maximum over the lanes; an fp32 image is
// shortened for it, and a token whose choice the shortened ones do not decide
// is chosen again from the whole ones.  Sums are fp32 in a fixed order.
// Bound by the integer and selection instructions of the rounds (65537 tokens x
// 128, top-8, fp32: forward 18.8 us over all experts, 17.4 over the chosen,
// gradient 10.6 us, 5.6 and 10.5 of memory; bf16 forward 16.1 and 14.7, 3.1 of
// memory).  Equal fp32 logits are not decided by shortened images either: of
// logits upcast from bf16 about every third token ties, 30.8 us for the 17.4.
// With 513 to 1024 experts of 16 bits some of a lane's 32 images spill (148 bytes
// a thread): 8192 x 1024 13.7 us, x 512 7.8; fp32 20.3 and 9.3.  The
// lane's sorted images in shared memory instead of registers, so that a round
// moves one of them: the same there, 0.2 us slower for few tokens.
#include "common.cuh"
#include "gate.cuh"
#include "launch.h"

namespace moeq {

namespace {

constexpr int kGateWarps = 4;

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

// The guard of a store to the logits' gradient.
template <int DT>
__device__ __forceinline__ bool grad_fits(const GateParams &p, const uint8_t *at, int bytes) {
    return store_fits(at, bytes, p.d_logits, p.num_tokens * p.E * kSize<DT>, p.err);
}

template <int DT, int NV>
__device__ __forceinline__ void store_row(const GateParams &p, uint8_t *row, int j0, bool vec,
                                          const float (&g)[NV]) {
    constexpr int kBytes = NV * kSize<DT>;
    if (vec && j0 + NV <= p.E && kBytes >= 8) {
        uint8_t *a = row + (int64_t)j0 * kSize<DT>;
        if (!grad_fits<DT>(p, a, kBytes)) return;
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
            if (j0 + i < p.E && grad_fits<DT>(p, row + (int64_t)(j0 + i) * kSize<DT>, kSize<DT>))
                store_logit<DT>(row, j0 + i, g[i]);
    }
}

// A lane's candidates as sorted images, each with its index in the low IB bits
// (largest first: the lowest index of equal ones).  A 16-bit logit is whole in
// what is left (fp16 needs 19 bits of an fp32 image), an fp32 one is shortened.
template <int DT, int NV, int L>
struct Candidates {
    static constexpr int log2(int v) { return v <= 1 ? 0 : 1 + log2(v / 2); }
    static constexpr int IB = log2(L * NV);
    static_assert(IB <= 10, "images of 16-bit logits are whole");
    static constexpr uint32_t kIdx = (1u << IB) - 1u;
    // the largest image of -inf; a NaN's is below kIdx
    static constexpr uint32_t kNone = kNegInfKey;
    uint32_t key[NV];
    // Odd-even merge sort, largest first (NV is a power of two): from the step
    // that compares keys h apart while runs of n are merged.
    template <int n, int h>
    __device__ __forceinline__ void merge_step() {
        if constexpr (n < NV) {
#pragma unroll
            for (int i = h % n; i + h < NV; ++i)
                if ((i - h % n) / h % 2 == 0 && i / (2 * n) == (i + h) / (2 * n)) {
                    const uint32_t u = key[i], v = key[i + h];
                    key[i] = max(u, v);
                    key[i + h] = min(u, v);
                }
            if constexpr (h > 1)
                merge_step<n, h / 2>();
            else
                merge_step<2 * n, 2 * n>();
        }
    }
    // nan: whether a logit of the warp is one
    __device__ __forceinline__ void init(const float (&x)[NV], int j0, bool nan) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            key[i] = (order_key(x[i]) & ~kIdx) | (kIdx - (uint32_t)(j0 + i));
        if (nan) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (x[i] != x[i]) key[i] &= kIdx;
        }
        merge_step<1, 1>();
    }
};

// The same choice from whole fp32 images, for a warp with a token whose
// shortened ones do not decide it: the token's lane r gets choice r (-1: none
// left) and its logit.
template <int NV, int L>
__device__ __forceinline__ void choose_exactly(const float (&x)[NV], int top_k, int lane,
                                               int &my_j, float &my_v) {
    const int sub = lane % L;
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = x[i] == x[i] ? order_key(x[i]) : 0u;
    for (int r = 0; r < top_k; ++r) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] > best) {  // the lowest index of equal ones
                best = key[i];
                at = i;
            }
        const uint32_t mx = lanes_max<L>(best);
        const uint32_t has = __ballot_sync(0xFFFFFFFFu, best == mx) >> (lane - sub);
        const int owner = __ffs((int)has) - 1;  // the token's first lane with it
        const int j = owner * NV + __shfl_sync(0xFFFFFFFFu, at, owner, L);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (sub == owner && i == at) key[i] = 0u;
        if (sub == r) {
            my_j = mx > kNegInfKey ? j : -1;
            my_v = key_value(mx);
        }
    }
}

// L lanes per token (top_k <= L), each with NV consecutive logits.
template <int DT, int NV, int L>
__global__ void __launch_bounds__(kGateWarps * 32) gate_kernel(GateParams p) {
    using Cand = Candidates<DT, NV, L>;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane % L;
    const int64_t warp = (int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5);
    const int64_t slot = warp * (32 / L) + lane / L;
    const bool active = slot < p.num_tokens;
    const int64_t t = active ? slot : p.num_tokens - 1;
    const uint8_t *row = p.logits + t * p.stride;
    float x[NV];
    load_row<DT>(row, p.E, sub * NV, rows_aligned<DT, NV>(p.stride), x);
    // a token's best images in the order of the rounds
    __shared__ uint32_t chosen[kGateWarps][32 / L][L + 1];
    uint32_t *out = chosen[threadIdx.x >> 5][lane / L];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) nan |= x[i] != x[i];
    Cand c;
    c.init(x, sub * NV, __any_sync(0xFFFFFFFFu, nan));
    // fp32: one round more than choices; where two rounds in a row find the same
    // image but for the index, the order is not decided
    const int rounds = p.top_k + (DT == MOEQ_FP32 ? 1 : 0);
    for (int r = 0; r < rounds; ++r) {
        const uint32_t mx = lanes_max<L>(c.key[0]);
        const bool own = c.key[0] == mx;  // one lane's while any image is left
        if (own) out[r] = mx;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            c.key[i] = own ? (i + 1 < NV ? c.key[(i + 1) % NV] : 0u) : c.key[i];
    }
    __syncwarp();
    uint32_t my_key = 0u;  // lane r of a token: choice r
    bool tie = false;
    if (sub < p.top_k) {
        my_key = out[sub];
        if constexpr (DT == MOEQ_FP32)
            tie = my_key > Cand::kNone && ((my_key ^ out[sub + 1]) >> Cand::IB) == 0u;
    }
    int id = -1;
    float v = 0.0f, w = 0.0f;
    if (my_key > Cand::kNone && sub < p.top_k) {
        id = (int)(Cand::kIdx - (my_key & Cand::kIdx));
        if constexpr (DT == MOEQ_FP32)
            v = load_logit<DT>(row, id);
        else
            v = __uint_as_float(__float_as_uint(key_value(my_key)) & ~Cand::kIdx);
    }
    if constexpr (DT == MOEQ_FP32)
        if (__any_sync(0xFFFFFFFFu, tie)) choose_exactly<NV, L>(x, p.top_k, lane, id, v);
    const float m = __shfl_sync(0xFFFFFFFFu, v, 0, L);
    const bool some = __shfl_sync(0xFFFFFFFFu, id, 0, L) >= 0;
    const float e = id >= 0 ? exp_diff(v, m) : 0.0f;
    // a NaN logit, or m infinite, makes either denominator NaN
    float total = e;
    if (p.normalize) {
        if (nan) total = __int_as_float(0x7FFFFFFF);
    } else {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) total = __fadd_rn(total, exp_diff(x[i], m));
    }
    total = lanes_sum<L>(total);
    if (some) w = __fmul_rn(__fdiv_rn(e, total), p.scale);
    if (active && sub < p.top_k) {
        int32_t *ids = p.ids + t * p.top_k + sub;
        float *weights = p.weights + t * p.top_k + sub;
        const int64_t size = p.num_tokens * p.top_k * 4;
        if (store_fits(ids, 4, p.ids, size, p.err)) *ids = id;
        if (store_fits(weights, 4, p.weights, size, p.err)) *weights = w;
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
    if (active) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float g[W];
#pragma unroll
            for (int k = 0; k < W; ++k) g[k] = p.normalize ? 0.0f : __fmul_rn(part, x[i][k]);
            store_row<DT>(p, out, (i * LANES + sub) * W, vec & 2, g);
        }
    }
    __syncwarp();  // orders the stores above before those below
    if (active && id >= 0 && grad_fits<DT>(p, out + id * kS, kSize<DT>))
        store_logit<DT>(out, id, __fmul_rn(q, __fadd_rn(d, -mean)));
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

template <int DT, int NV, int L>
cudaError_t run_gate_lanes(const GateParams &p, cudaStream_t s) {
    const int64_t per_cta = kGateWarps * 32 / L;
    return launch_pdl(gate_kernel<DT, NV, L>, (unsigned)((p.num_tokens + per_cta - 1) / per_cta),
                      kGateWarps * 32, 0, s, p);
}

template <int DT>
cudaError_t run_gate(const GateParams &p, cudaStream_t s) {
    // many tokens: as few lanes per token as leave each at most 8 logits, so that
    // the rounds of a warp's tokens are shared.  fp32, top-8, normalised, these
    // lanes against 32: 65536 tokens x 32 experts 6.7 / 17.8 us, x 64 8.5 / 17.9, x
    // 128 17.4 / 20.3; 16384 x 128 6.2 / 6.3 (bf16 5.5 / 5.7), 8192 x 64 3.2 / 3.7, x
    // 128 5.1 / 4.3; 4096 x 64 3.0 / 2.6
    if (p.num_tokens >= 8192 && p.top_k <= 8) {
        if (p.E <= 32) return run_gate_lanes<DT, 4, 8>(p, s);
        if (p.E <= 64) return run_gate_lanes<DT, 8, 8>(p, s);
    }
    if (p.num_tokens >= 16384 && p.E <= 128 && p.top_k <= 16)
        return run_gate_lanes<DT, 8, 16>(p, s);
    const int nv = (p.E + 31) / 32;
    return nv <= 1    ? run_gate_lanes<DT, 1, 32>(p, s)
           : nv <= 2  ? run_gate_lanes<DT, 2, 32>(p, s)
           : nv <= 4  ? run_gate_lanes<DT, 4, 32>(p, s)
           : nv <= 8  ? run_gate_lanes<DT, 8, 32>(p, s)
           : nv <= 16 ? run_gate_lanes<DT, 16, 32>(p, s)
                      : run_gate_lanes<DT, 32, 32>(p, s);
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
