// The router with scores, a balance bias and groups of experts.  With x the
// logits of a token, s_j = sigmoid(x_j) or softmax(x)_j and b the bias:
//
//   c_j = s_j + b_j                       decides the choice, not the weights
//   a group's value: its best c, or the sum of its best two
//   i_1 .. i_k: the best c in the best topk_groups groups (ties: lowest index)
//   w_r = scale s_{i_r}                   or, normalised,
//   w_r = scale s_{i_r} / sum over the choices of s
//
// and, the choice fixed, with q = w / scale and g_r = scale d_w_r,
//
//   d_x_{i_r} = g_r s (1 - s)                        sigmoid
//   d_x_{i_r} = q_r (g_r - <q, g>) (1 - s)           sigmoid, normalised
//   d_x_{i_r} = q_r (g_r - <q, g>)                   softmax, normalised
//
// and 0 elsewhere (plain softmax: the gradient of the router over all experts,
// gate.cu).
//
// The row of a token is in the registers of L lanes, a power of two of them for
// each group (lane and index order are expert order), read once.  Keys are the
// bits of max c - c with the lane and index in the low bits: those of the best
// values, close to the maximum, keep most of their digits, so that a round of the
// choice is one integer minimum over the lanes.  Scores next to one another are
// decided in 64 bits: c in fp32 is off by a bound known beforehand, and a token
// in which two values that the choice depends on are closer than that (about one
// in a thousand) is chosen again from 64-bit scores.
#include <algorithm>

#include "common.cuh"
#include "gate.cuh"
#include "launch.h"

namespace moeq {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxPerLane = 32;

struct ScoredParams {
    const uint8_t *logits;
    int64_t stride;  // bytes
    int64_t num_tokens;
    int E, top_k;
    const float *bias;  // null: none
    int sigmoid, top2, normalize;
    int groups, topk_groups;
    int group_size, lane_shift, per_lane;  // 1 << lane_shift lanes a group, per_lane logits each
    int vec;                               // a lane's logits are aligned vectors
    float scale;
    int32_t *ids;
    float *weights;
    uint32_t *err;
};

// 1 / (1 + exp(-x)) within 4e-7: exp is within 2 + 1.2 |x| ulp of 2^-23, which
// s (1 - s) turns into 8e-8 at most; the sum and the quotient (2 ulp) add 3e-7 s.
__device__ __forceinline__ float score_fast(float x) {
    return __fdividef(1.0f, __fadd_rn(1.0f, __expf(-x)));
}

constexpr float kScoreTol = 4e-7f;

// A softmax's p, relative: exp's 2 + 1.2 |d| ulp (at most 2 ulp of the largest p),
// the total's own error, the mean of its terms' (ln 1024 bounds the mean of |d|) and
// (32 + 5) 2^-24 of its sums, and the product's: 4e-6 of the largest p.
constexpr float kSoftmaxTol = 5e-6f;

// sigmoid(x) for the weights: within a few ulp of either end.
__device__ __forceinline__ float sigmoid_exact(float x) {
    const float e = expf(-fabsf(x));
    return __fdiv_rn(x >= 0.0f ? 1.0f : e, __fadd_rn(1.0f, e));
}

template <int L>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
    if constexpr (L == 32) return __reduce_min_sync(0xFFFFFFFFu, v);
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v = min(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

__device__ __forceinline__ float load_any(const uint8_t *row, int j, int dt) {
    return dt == MOEQ_FP32 ? load_logit<MOEQ_FP32>(row, j)
           : dt == MOEQ_BF16 ? load_logit<MOEQ_BF16>(row, j)
                             : load_logit<MOEQ_FP16>(row, j);
}

// The place of a lane: its first expert, how many it holds, its group.
struct Place {
    int j0, n, group;
};

__device__ __forceinline__ Place place_of(const ScoredParams &p, int sub) {
    Place a;
    a.group = sub >> p.lane_shift;
    const int at = (sub & ((1 << p.lane_shift) - 1)) * p.per_lane;
    a.n = a.group < p.groups ? max(0, min(p.per_lane, p.group_size - at)) : 0;
    a.j0 = a.group * p.group_size + at;
    return a;
}

// Best two of pairs (a >= b) and (c >= d).
template <class T>
__device__ __forceinline__ void best_two(T &a, T &b, T c, T d) {
    b = a < c ? (a > d ? a : d) : (b > c ? b : c);
    a = a > c ? a : c;
}

template <class T>
__device__ __forceinline__ T group_value(T a, T b, bool sum, T none) {
    return sum && b > none ? a + b : a;
}

// The choice from 64-bit scores, for a warp with a token that 32 bits do not
// decide; lane r of each token gets choice r (-1: none left).
__device__ __noinline__ int choose_64(const ScoredParams &p, const uint8_t *row, int dt, int lane,
                                      int L) {
    constexpr unsigned kAll = 0xFFFFFFFFu;
    const double none = -__longlong_as_double(0x7FF0000000000000ll);
    const int sub = lane % L;
    const Place a = place_of(p, sub);
    double c[kMaxPerLane];
    float m = -kInf;
    int bad = 0;
    for (int i = 0; i < a.n; ++i) {
        const float x = load_any(row, a.j0 + i, dt);
        bad |= x != x;
        m = fmaxf(m, x);
        c[i] = x > -kInf ? (double)x : none;
    }
    for (int o = L / 2; o; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        bad |= __shfl_xor_sync(kAll, bad, o);
    }
    const bool plain = !p.sigmoid && (bad || m == kInf);  // no softmax: by the logits
    double total = 0.0;
    if (!p.sigmoid) {
        for (int i = 0; i < a.n; ++i)
            if (c[i] > none) total += exp(c[i] - (double)m);
        for (int o = L / 2; o; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    }
    const bool by_score = !plain && (p.bias || (p.groups > 1 && p.top2));
    double g1 = none, g2 = none;
    for (int i = 0; i < a.n; ++i) {
        double v = c[i];
        if (by_score && c[i] > none) {
            v = p.sigmoid ? 1.0 / (1.0 + exp(-c[i])) : exp(c[i] - (double)m) / total;
            if (p.bias) {
                v += (double)__ldg(p.bias + a.j0 + i);
                c[i] = v = v > none ? v : none;
            }
        }
        best_two(g1, g2, v, none);
    }
    if (p.groups > 1) {
        for (int o = (1 << p.lane_shift) / 2; o; o >>= 1) {
            const double b1 = __shfl_xor_sync(kAll, g1, o), b2 = __shfl_xor_sync(kAll, g2, o);
            best_two(g1, g2, b1, b2);
        }
        const double v = group_value(g1, g2, p.top2 && !plain, none);
        int rank = 0;
        for (int h = 0; h < p.groups; ++h) {
            const double u = __shfl_sync(kAll, v, h << p.lane_shift, L);
            rank += u > v || (u == v && h < a.group);
        }
        if (rank >= p.topk_groups)
            for (int i = 0; i < a.n; ++i) c[i] = none;
    }
    int id = -1;
    uint32_t taken = 0u;
    for (int r = 0; r < p.top_k; ++r) {
        double best = none;
        int at = 0x7FFFFFFF;
        for (int i = 0; i < a.n; ++i)
            if (!((taken >> i) & 1u) && c[i] > best) {
                best = c[i];
                at = a.j0 + i;
            }
        for (int o = L / 2; o; o >>= 1) {
            const double v = __shfl_xor_sync(kAll, best, o);
            const int j = __shfl_xor_sync(kAll, at, o);
            if (v > best || (v == best && j < at)) {
                best = v;
                at = j;
            }
        }
        if (at >= a.j0 && at < a.j0 + a.n) taken |= 1u << (at - a.j0);
        if (sub == r) id = best > none ? at : -1;
    }
    return id;
}

// Keys sorted smallest first by an odd-even merge (NV is a power of two).
template <int NV, int n, int h>
__device__ __forceinline__ void merge_step(uint32_t (&key)[NV]) {
    if constexpr (n < NV) {
#pragma unroll
        for (int i = h % n; i + h < NV; ++i)
            if ((i - h % n) / h % 2 == 0 && i / (2 * n) == (i + h) / (2 * n)) {
                const uint32_t u = key[i], v = key[i + h];
                key[i] = min(u, v);
                key[i + h] = max(u, v);
            }
        if constexpr (h > 1)
            merge_step<NV, n, h / 2>(key);
        else
            merge_step<NV, 2 * n, 2 * n>(key);
    }
}

template <int DT, int NV, int L>
__global__ void __launch_bounds__(kWarps * 32) gate_scored_kernel(ScoredParams p) {
    constexpr unsigned kAll = 0xFFFFFFFFu;
    constexpr uint32_t kIdx = (uint32_t)(L * NV) - 1u, kNoKey = 0xFFFFFFFFu;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane % L;
    const int64_t slot =
        ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * (32 / L) + lane / L;
    const bool active = slot < p.num_tokens;
    const int64_t t = active ? slot : p.num_tokens - 1;
    const uint8_t *row = p.logits + t * p.stride;
    const Place a = place_of(p, sub);
    float x[NV];
    load_row<DT>(row, a.j0 + a.n, a.j0, p.vec, x);
    // c, -inf for what is never chosen
    float c[NV], m = -kInf, inv = 0.0f, total = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        nan |= x[i] != x[i];
        m = fmaxf(m, x[i]);
    }
    bool plain = false;
    if (!p.sigmoid) {
#pragma unroll
        for (int o = L / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (m > -kInf) {
#pragma unroll
            for (int i = 0; i < NV; ++i) total = __fadd_rn(total, exp_diff(x[i], m));
        }
        total = lanes_sum<L>(total);
        inv = __fdividef(1.0f, total);
        plain = !(total < kInf);  // NaN: a NaN logit, or m infinite
    }
    auto score = [&](float v) {
        return p.sigmoid ? score_fast(v) : __fmul_rn(exp_diff(v, m), inv);
    };
    // c of a logit and its bias
    auto value = [&](float v, float b) {
        return p.bias && !plain ? __fadd_rn(score(v), b) : v;
    };
    // how far apart two values are decided: twice the scores' bound, and the
    // rounding of the sums with the bias (2^-24 each, taken as 2^-22)
    const float tol =
        plain ? 0.0f : 2.0f * (p.sigmoid ? kScoreTol : __fmul_rn(kSoftmaxTol, inv));
    bool unsure = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float b = p.bias && i < a.n ? __ldg(p.bias + a.j0 + i) : 0.0f;
        const float v = value(x[i], b);
        c[i] = x[i] > -kInf && v > -kInf ? v : -kInf;
    }
    if (p.groups > 1) {
        const bool sum = p.top2 && !plain, scores = sum && !p.bias;
        float g1 = -kInf, g2 = -kInf;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            best_two(g1, g2, scores && c[i] > -kInf ? score(c[i]) : c[i], -kInf);
        for (int o = (1 << p.lane_shift) / 2; o; o >>= 1) {
            const float b1 = __shfl_xor_sync(kAll, g1, o), b2 = __shfl_xor_sync(kAll, g2, o);
            best_two(g1, g2, b1, b2);
        }
        const float v = group_value(g1, g2, sum, -kInf);
        // twice the error of this group's value, so that of two the larger counts
        const float size = __fadd_rn(fabsf(g1), sum && g2 > -kInf ? fabsf(g2) : 0.0f);
        const float near = (sum || p.bias) && !plain
                               ? __fadd_rn(2.0f * tol, __fmul_rn(size, 0x1p-20f))
                               : -1.0f;
        int rank = 0;
        float above = kInf, below = -kInf;  // the nearest groups' values
        for (int h = 0; h < p.groups; ++h) {
            const float u = __shfl_sync(kAll, v, h << p.lane_shift, L);
            const bool ahead = u > v || (u == v && h < a.group);
            rank += ahead;
            if (ahead) above = fminf(above, u);
            if (!ahead && h != a.group) below = fmaxf(below, u);
        }
        // only the border between the chosen groups and the others counts
        if (a.n > 0 && v > -kInf) {
            if (rank == p.topk_groups) unsure = above - v <= near;
            if (rank == p.topk_groups - 1) unsure = v - below <= near;
        }
        if (rank >= p.topk_groups) {
#pragma unroll
            for (int i = 0; i < NV; ++i) c[i] = -kInf;
        }
    }
    float top = -kInf;
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, c[i]);
#pragma unroll
    for (int o = L / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        // an infinite c is as far from itself as 0
        const float d = c[i] == top ? 0.0f : __fadd_rn(top, -c[i]);
        key[i] = c[i] > -kInf ? (__float_as_uint(d) & ~kIdx) | (uint32_t)(sub * NV + i) : kNoKey;
    }
    merge_step<NV, 1, 1>(key);
    // a token's best keys, and the one behind them
    __shared__ uint32_t chosen[kWarps][32 / L][L + 1];
    uint32_t *out = chosen[threadIdx.x >> 5][lane / L];
    for (int r = 0; r <= p.top_k; ++r) {
        const uint32_t mn = lanes_min<L>(key[0]);
        const bool own = key[0] == mn;
        if (own) out[r] = mn;
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = own ? (i + 1 < NV ? key[(i + 1) % NV] : kNoKey) : key[i];
    }
    __syncwarp();
    auto expert_of = [&](uint32_t k) {
        const Place b = place_of(p, (int)((k & kIdx) / NV));
        return b.j0 + (int)(k & kIdx) % NV;
    };
    // whether a key that differs from the one behind the choices by its index alone is
    // left: its c can be above by the width of what the index took
    const uint32_t last = out[p.top_k];
    const bool hidden = ((lanes_min<L>(key[0]) ^ last) & ~kIdx) == 0u;
    int id = -1;
    float v = 0.0f, b = 0.0f, cv = -kInf;
    if (sub <= p.top_k && out[sub] != kNoKey) {
        id = expert_of(out[sub]);
        v = load_logit<DT>(row, id);
        if (p.bias) b = __ldg(p.bias + id);
        cv = value(v, b);
    }
    float vn = __shfl_down_sync(kAll, v, 1, L), bn = __shfl_down_sync(kAll, b, 1, L);
    float cn = __shfl_down_sync(kAll, cv, 1, L);
    if (sub == L - 1 && p.top_k == L) {
        cn = -kInf;
        if (last != kNoKey) {
            const int j = expert_of(last);
            vn = load_logit<DT>(row, j);
            if (p.bias) bn = __ldg(p.bias + j);
            cn = value(vn, bn);
        }
    }
    const bool border = sub == p.top_k - 1 && hidden;
    // the same logit and bias: the lower index is first
    if (sub < p.top_k && id >= 0 && cn > -kInf && (border || v != vn || b != bn)) {
        float near = p.bias && !plain
                         ? __fadd_rn(tol, __fmul_rn(fmaxf(fabsf(cv), fabsf(cn)), 0x1p-22f))
                         : 0.0f;
        if (border) near = __fadd_rn(near, __fmul_rn(__fadd_rn(top, -cn), (kIdx + 1u) * 0x1p-22f));
        unsure |= !(__fadd_rn(cv, -cn) > near);
    }
    if (sub >= p.top_k) id = -1;
    if (__any_sync(kAll, unsure)) {
        id = choose_64(p, row, DT, lane, L);
        if (id >= 0) v = load_logit<DT>(row, id);
    }
    // the weights
    const bool some = __shfl_sync(kAll, id, 0, L) >= 0;
    float s = 0.0f, sum = 0.0f;
    if (p.sigmoid) {
        if (id >= 0) s = sigmoid_exact(v);
        sum = p.normalize ? s : 1.0f;
    } else if (p.normalize) {
        // relative to the largest of the chosen
        float mc = id >= 0 ? v : -kInf;
#pragma unroll
        for (int o = L / 2; o; o >>= 1) mc = fmaxf(mc, __shfl_xor_sync(kAll, mc, o));
        if (id >= 0) s = exp_diff(v, mc);
        sum = s;
    } else {
        if (id >= 0) s = exp_diff(v, m);
    }
    if (p.normalize) sum = lanes_sum<L>(sum);
    if (!p.sigmoid && !p.normalize) sum = total;
    // a NaN, or an infinity in a softmax, is seen in all of the token's weights
#pragma unroll
    for (int o = L / 2; o; o >>= 1) nan |= __shfl_xor_sync(kAll, (int)nan, o) != 0;
    float w = sum > 0.0f ? __fmul_rn(__fdiv_rn(s, sum), p.scale) : 0.0f;
    if (nan || plain) w = __int_as_float(0x7FFFFFFF);
    if (!some) w = 0.0f;
    if (active && sub < p.top_k) {
        int32_t *ids = p.ids + t * p.top_k + sub;
        float *weights = p.weights + t * p.top_k + sub;
        const int64_t size = p.num_tokens * p.top_k * 4;
        if (store_fits(ids, 4, p.ids, size, p.err)) *ids = id;
        if (store_fits(weights, 4, p.weights, size, p.err)) *weights = w;
    }
}

struct ChosenGradParams {
    const uint8_t *logits;
    int64_t stride;  // bytes
    int64_t num_tokens;
    int E, top_k;
    int sigmoid, normalize;
    float scale;
    const int32_t *ids;
    const float *d_weights;
    uint8_t *d_logits;
    int vec;  // rows of d_logits are whole 16-byte vectors
    uint32_t *err;
};

// The gradient that only the chosen logits have: LANES lanes a token (top_k <=
// LANES).  The row is zeroed first, the choices stored over it.
template <int DT, int LANES>
__global__ void __launch_bounds__(kWarps * 32) gate_chosen_grad_kernel(ChosenGradParams p) {
    pdl_wait();
    pdl_trigger();
    constexpr int64_t kS = kSize<DT>;
    const int lane = threadIdx.x & 31, sub = lane % LANES;
    const int64_t slot = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * (32 / LANES) +
                         lane / LANES;
    const bool active = slot < p.num_tokens;
    const int64_t t = active ? slot : p.num_tokens - 1;
    const uint8_t *in = p.logits + t * p.stride;
    uint8_t *out = p.d_logits + t * p.E * kS;
    const int64_t size = p.num_tokens * p.E * kS;
    int id = -1;
    float g = 0.0f, x = -kInf;
    if (sub < p.top_k) {
        id = __ldg(p.ids + t * p.top_k + sub);
        if (id < -1 || id >= p.E) {
            if (active) set_error(p.err, MOEQ_DEVERR_BAD_EXPERT);
            id = -1;
        }
        if (id >= 0) {
            g = __fmul_rn(__ldg(p.d_weights + t * p.top_k + sub), p.scale);
            x = load_logit<DT>(in, id);
        }
    }
    if (active) {
        if (p.vec) {
            for (int64_t at = sub * 16; at < p.E * kS; at += LANES * 16)
                if (store_fits(out + at, 16, p.d_logits, size, p.err))
                    st_global_v4(out + at, 0u, 0u, 0u, 0u);
        } else {
            for (int j = sub; j < p.E; j += LANES)
                if (store_fits(out + j * kS, kS, p.d_logits, size, p.err))
                    store_logit<DT>(out, j, 0.0f);
        }
    }
    float d = 0.0f;
    if (p.sigmoid) {
        const float s = id >= 0 ? sigmoid_exact(x) : 0.0f;
        const float rest = sigmoid_exact(-x);
        if (p.normalize) {
            const float total = lanes_sum<LANES>(s);
            const float q = total > 0.0f ? __fdiv_rn(s, total) : total == 0.0f ? 0.0f : total;
            const float mean = lanes_sum<LANES>(__fmul_rn(q, g));
            d = __fmul_rn(__fmul_rn(q, __fadd_rn(g, -mean)), rest);
        } else {
            d = __fmul_rn(__fmul_rn(g, s), rest);
        }
    } else {
        float m = x;
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float e = id >= 0 ? expf(__fadd_rn(x, -m)) : 0.0f;
        const float total = lanes_sum<LANES>(e);
        const float q = id >= 0 ? __fdiv_rn(e, total) : 0.0f;
        const float mean = lanes_sum<LANES>(__fmul_rn(q, g));
        d = __fmul_rn(q, __fadd_rn(g, -mean));
    }
    __syncwarp();  // orders the zeros before the choices
    if (active && id >= 0 && store_fits(out + id * kS, kS, p.d_logits, size, p.err))
        store_logit<DT>(out, id, d);
}

template <int DT, int NV, int L>
cudaError_t run_lanes(const ScoredParams &p, cudaStream_t s) {
    const int64_t per_cta = kWarps * 32 / L;
    return launch_pdl(gate_scored_kernel<DT, NV, L>,
                      (unsigned)((p.num_tokens + per_cta - 1) / per_cta), kWarps * 32, 0, s, p);
}

// The lanes and logits per lane of a token's groups on L lanes; false where a
// lane would hold more than kMaxPerLane.
bool lay_out(ScoredParams &p, int L, int size) {
    int lanes = L;  // of a group
    while (lanes > 0 && lanes * p.groups > L) lanes /= 2;
    if (lanes == 0) return false;
    p.group_size = p.E / p.groups;
    p.per_lane = (p.group_size + lanes - 1) / lanes;
    if (p.per_lane > kMaxPerLane) return false;
    p.lane_shift = 0;
    while ((1 << p.lane_shift) < lanes) ++p.lane_shift;
    int nv = 1;
    while (nv < p.per_lane) nv *= 2;
    if (p.groups == 1) p.per_lane = nv;  // whole vectors
    const int bytes = std::min(nv * size, 16);
    p.vec = p.per_lane == nv && p.stride % bytes == 0 && p.group_size * size % bytes == 0;
    if (p.groups == 1) p.vec = p.stride % bytes == 0;
    return true;
}

template <int DT>
cudaError_t run_scored(ScoredParams p, cudaStream_t s) {
    if (!lay_out(p, 32, kSize<DT>)) return cudaErrorNotSupported;
    return p.per_lane <= 1    ? run_lanes<DT, 1, 32>(p, s)
           : p.per_lane <= 2  ? run_lanes<DT, 2, 32>(p, s)
           : p.per_lane <= 4  ? run_lanes<DT, 4, 32>(p, s)
           : p.per_lane <= 8  ? run_lanes<DT, 8, 32>(p, s)
           : p.per_lane <= 16 ? run_lanes<DT, 16, 32>(p, s)
                              : run_lanes<DT, 32, 32>(p, s);
}

template <int DT>
cudaError_t run_grad(ChosenGradParams p, cudaStream_t s) {
    p.vec = p.E * kSize<DT> % 16 == 0;
    auto go = [&](void (*kern)(ChosenGradParams), int lanes) {
        const int64_t per_cta = kWarps * 32 / lanes;
        return launch_pdl(kern, (unsigned)((p.num_tokens + per_cta - 1) / per_cta), kWarps * 32, 0,
                          s, p);
    };
    if (p.top_k <= 8) return go(gate_chosen_grad_kernel<DT, 8>, 8);
    return go(gate_chosen_grad_kernel<DT, 32>, 32);
}

}  // namespace

cudaError_t launch_gate_scored(const GateScoredArgs &a, cudaStream_t s) {
    const int64_t size = a.dtype == MOEQ_FP32 ? 4 : 2;
    ScoredParams p = {};
    p.logits = static_cast<const uint8_t *>(a.logits);
    p.stride = a.stride * size;
    p.num_tokens = a.num_tokens;
    p.E = a.num_experts;
    p.top_k = a.top_k;
    p.bias = a.bias;
    p.sigmoid = a.sigmoid;
    p.top2 = a.top2;
    p.normalize = a.normalize;
    p.groups = a.groups;
    p.topk_groups = a.topk_groups;
    p.scale = a.scale;
    p.ids = a.ids;
    p.weights = a.weights;
    p.err = a.err;
    if (a.dtype == MOEQ_BF16) return run_scored<MOEQ_BF16>(p, s);
    if (a.dtype == MOEQ_FP16) return run_scored<MOEQ_FP16>(p, s);
    return run_scored<MOEQ_FP32>(p, s);
}

cudaError_t launch_gate_chosen_grad(const GateArgs &a, bool sigmoid, cudaStream_t s) {
    const int64_t size = a.dtype == MOEQ_FP32 ? 4 : 2;
    const ChosenGradParams p{static_cast<const uint8_t *>(a.logits), a.stride * size, a.num_tokens,
                             a.num_experts, a.top_k, sigmoid, a.normalize, a.scale, a.ids,
                             a.d_weights, static_cast<uint8_t *>(a.d_logits), 0, a.err};
    if (a.dtype == MOEQ_BF16) return run_grad<MOEQ_BF16>(p, s);
    if (a.dtype == MOEQ_FP16) return run_grad<MOEQ_FP16>(p, s);
    return run_grad<MOEQ_FP32>(p, s);
}

}  // namespace moeq
