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
// bits of max c - c with the lane and index in the low bits (of 16-bit logits without
// a bias: their whole images): those of the best values, close to the maximum, keep
// most of their digits, so that a round of the choice is one integer minimum over the
// lanes.  Scores next to one another are decided as the reals would: c in fp32 is off by
// a bound known beforehand, and a token in which two values that the choice depends on
// are closer than that (about one in a thousand) looks at those again as sums of two
// floats (within 2^-44).
//
// Bound by a token's chain of dependent steps: no pipe is full (that of integer minima and
// comparisons 42 %, the issue slots 58 %) at four warps a scheduler, which a CTA of 16 tokens
// leaves with its bias, rows and barrier before it to wait for.  Some 370 instructions a
// token of 256 experts.  65537 x 256, 8
// groups of which 4, top-8, sigmoid and bias: forward 35 us fp32, 33 bf16 (10 and 5 of
// memory), gradient 15 (10); 65536 x 128, one group, top-4, 18; 9999 x 160 softmax, 8
// groups, top-6, 7.6; 64 x 256 2.9.  A token that is looked at again takes 3 us more (in
// 64-bit floats 7 to 40), in time with the others'.  More CTAs on an SM by fewer
// registers: none faster, 8 of them 15 % slower.
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
    int dt, E, top_k;
    const float *bias;  // null: none
    int sigmoid, top2, normalize;
    int groups, topk_groups;
    int group_size, lane_shift, per_lane;  // 1 << lane_shift lanes a group, per_lane logits each
    int vec, bias_vec;                     // a lane's logits, biases are aligned vectors
    int staged;                            // and the lanes' are the whole row, in order
    int halves;                            // a group is a lane, at most half of them are chosen
    float scale;
    int32_t *ids;
    float *weights;
    uint32_t *err;
};

// exp and sigma of fp32 by 2^x and 1 / x of the hardware, results below 2^-126 as 0.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-x)) within kScoreTol: exp is within 2^-22 + |x| 2^-23 relative, which
// s (1 - s) turns into 8e-8 at most; the sum and the quotient add 2e-7 s.
__device__ __forceinline__ float score_fast(float x) {
    return rcp_fast(__fadd_rn(1.0f, exp2_fast(__fmul_rn(x, -kLog2e))));
}
constexpr float kScoreTol = 4e-7f;

// exp(x - m), x <= m, within 2^-22 + |x - m| 2^-22 relative (the difference and its
// product are rounded).
__device__ __forceinline__ float exp_fast(float x, float m) {
    return exp2_fast(__fmul_rn(__fadd_rn(x, -m), kLog2e));
}
// A softmax's p, in units of the largest one: 2 2^-22 of it for exp, and relative the
// total's own error, the mean of its terms' (ln 1024 bounds the mean of |x - m|), (32 + 5)
// 2^-24 of its sums and 2^-22 of the quotient: 4.9e-6.
constexpr float kSoftmaxTol = 5e-6f;
// without the total, exp alone
constexpr float kExpTol = 6e-7f;

// sigmoid(x) for the weights: within 4 ulp at either end (exp 2, the sum half, 1 / x one
// and the product half).
__device__ __forceinline__ float sigmoid_exact(float x) {
    const float e = expf(-fabsf(x));
    return __fmul_rn(x >= 0.0f ? 1.0f : e, rcp_fast(__fadd_rn(1.0f, e)));
}

template <int L>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
    if constexpr (L == 32) return __reduce_min_sync(0xFFFFFFFFu, v);
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v = min(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// The largest of the lanes' floats, none a NaN.
template <int L>
__device__ __forceinline__ float lanes_top(float v) {
    if constexpr (L == 32) return key_value(lanes_max<L>(order_key(v)));
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
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

// The best two of a >= b and c >= d.
template <class T>
__device__ __forceinline__ void best_two(T &a, T &b, T c, T d) {
    const T lo = a < c ? a : c, hi = b > d ? b : d;
    a = a > c ? a : c;
    b = lo > hi ? lo : hi;
}

// What follows down to the kernel runs for one token in a thousand.  Fetching its
// instructions is much of what it costs, so that loops stay loops; 64-bit floats, which
// this machine takes some 90 cycles for, are left out (with them a pair of values took
// 13500 cycles and the groups 80000).

// A value as the sum of two floats, the second below half a unit of the first.
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair quick_sum(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fadd_rn(b, -__fadd_rn(s, -a))};
}
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), v = __fadd_rn(s, -a);
    return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -v)), __fadd_rn(b, -v))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const Pair s = two_sum(a.hi, b.hi);
    return quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    const float p = __fmul_rn(a.hi, b.hi);
    const float e = __fmaf_rn(a.hi, b.hi, -p);
    return quick_sum(p, __fadd_rn(e, __fmaf_rn(a.hi, b.lo, __fmul_rn(a.lo, b.hi))));
}
// 1 / d by a Newton step from 2^-23, with the step's square
__device__ __forceinline__ Pair reciprocal(Pair d) {
    const float r = rcp_fast(d.hi);
    const float e = __fmaf_rn(-d.lo, r, __fmaf_rn(-d.hi, r, 1.0f));
    return quick_sum(r, __fmul_rn(r, __fmaf_rn(e, e, e)));
}

// exp(x), x <= 0, within 2^-44: 2^n e^f with n = x / ln 2 to the nearest, ln 2 in three
// parts of which the first leaves n times it exact, and the Taylor series of e^f, |f| <=
// 0.35, to the 13th power (from the 8th on, below 2^-22 of the sum, in fp32).
__device__ __noinline__ Pair exp_pair(Pair x) {
    const float n = rintf(__fmul_rn(x.hi, kLog2e));
    if (!(n >= -126.0f)) return {0.0f, 0.0f};
    Pair f = two_sum(__fmaf_rn(n, -0x1.62ep-1f, x.hi), x.lo);
    f = add(f, mul({-n, 0.0f}, {0x1.0bfbe8p-15f, 0x1.cf79acp-40f}));
    float q = 1.0f, k = 13.0f;
#pragma unroll 1
    for (; k > 7.0f; k -= 1.0f) q = __fmaf_rn(__fmul_rn(q, f.hi), rcp_fast(k), 1.0f);
    Pair p = {q, 0.0f};
#pragma unroll 1
    for (; k > 0.0f; k -= 1.0f) p = add({1.0f, 0.0f}, mul(mul(p, f), reciprocal({k, 0.0f})));
    const float scale = __uint_as_float((uint32_t)((int)n + 127) << 23);
    return {__fmul_rn(p.hi, scale), __fmul_rn(p.lo, scale)};
}

// Integers that order as values do; 0 stands for none.  The second part is rounded to
// what 64-bit floats keep beside the first, so that what they cannot tell apart is equal.
__device__ __forceinline__ uint64_t pair_key(Pair v) {
    const float unit =
        __fmul_rn(__uint_as_float(__float_as_uint(v.hi) & 0x7F800000u), 1.5f * 0x1p-29f);
    const float lo = __fadd_rn(__fadd_rn(v.lo, unit), -unit);
    return ((uint64_t)order_key(v.hi) << 32) | order_key(lo);
}
__device__ __forceinline__ uint64_t float_key(float v) {
    return v > -kInf ? ((uint64_t)order_key(v) << 32) | 0x80000000u : 0u;
}
__device__ __forceinline__ float key_hi(uint64_t k) { return key_value((uint32_t)(k >> 32)); }
__device__ __forceinline__ Pair key_pair(uint64_t k) { return {key_hi(k), key_value((uint32_t)k)}; }
// half of the sum of two values, which cannot overflow; the second may be none, an infinite
// first one stays.  (In line, 65537 x 512 took 1.8 % longer.)
__device__ __noinline__ uint64_t half_sum_key(uint64_t a, uint64_t b) {
    if (a == 0u || !(key_hi(a) < kInf)) return a;
    const Pair u = key_pair(a), v = b != 0u ? key_pair(b) : Pair{0.0f, 0.0f};
    return pair_key(add({0.5f * u.hi, 0.5f * u.lo}, {0.5f * v.hi, 0.5f * v.lo}));
}

// What the calls below know of a token: its largest logit, whether its order is that of
// the logits (no bias, or no softmax), and the bound of the scores' errors, doubled.
struct Token {
    float m;
    bool plain;
    float tol;
};

// The sum of exp(x - m) over a token's logits.
__device__ __noinline__ Pair total_pair(const ScoredParams &p, const uint8_t *row, int lane, int L,
                                        float m) {
    const Place a = place_of(p, lane % L);
    Pair total = {0.0f, 0.0f};
#pragma unroll 1
    for (int i = 0; i < a.n; ++i) {
        const float x = load_any(row, a.j0 + i, p.dt);
        if (x > -kInf) total = add(total, exp_pair(two_sum(x, -m)));
    }
#pragma unroll 1
    for (int o = L / 2; o; o >>= 1)
        total = add(total, {__shfl_xor_sync(0xFFFFFFFFu, total.hi, o),
                            __shfl_xor_sync(0xFFFFFFFFu, total.lo, o)});
    return total;
}

// The key of c from a logit and its bias; of a softmax with its total.
__device__ __noinline__ uint64_t value_key(bool sigmoid, float x, float b, float m, Pair total) {
    // sigma by e = exp(-|x|): 1 / (1 + e) or e / (1 + e)
    const Pair e = exp_pair(sigmoid ? Pair{-fabsf(x), 0.0f} : two_sum(x, -m));
    const Pair r = reciprocal(sigmoid ? add({1.0f, 0.0f}, e) : total);
    return pair_key(add(sigmoid && x >= 0.0f ? r : mul(e, r), {b, 0.0f}));
}

// Keys of a lane's values in fp32 (none for what is never chosen) and which of them are
// final.  scored: c, or the sums' terms; else the logits.
__device__ __noinline__ uint32_t first_keys(const ScoredParams &p, const uint8_t *row, Place a,
                                            Token k, bool bias, bool scored, float total,
                                            uint64_t *c) {
    uint32_t known = scored ? 0u : 0xFFFFFFFFu;
#pragma unroll 1
    for (int i = 0; i < a.n; ++i) {
        const float x = load_any(row, a.j0 + i, p.dt);
        float v = x;
        if (scored) v = p.sigmoid ? score_fast(x) : __fdividef(exp_fast(x, k.m), total);
        if (bias) v = __fadd_rn(v, __ldg(p.bias + a.j0 + i));
        c[i] = x > -kInf ? float_key(v) : 0u;
        if (!(fabsf(v) < 1e30f)) known |= 1u << i;
    }
    return known;
}

__device__ __forceinline__ uint64_t shfl_xor_key(uint64_t k, int o) {
    return __shfl_xor_sync(0xFFFFFFFFu, (unsigned long long)k, o);
}

// The groups chosen, for a warp with a token whose fp32 values do not decide them:
// whether the lane's is.  Where the border between the chosen and the others depends
// on two values that are closer than their errors, what they sum is computed as pairs,
// and the groups are ranked again.
__device__ __noinline__ bool groups_again(const ScoredParams &p, const uint8_t *row, int lane,
                                          int L, Token k) {
    constexpr unsigned kAll = 0xFFFFFFFFu;
    const int sub = lane % L;
    const Place a = place_of(p, sub);
    const bool bias = p.bias && !k.plain, sums = p.top2 && !k.plain, scored = bias || sums;
    // the sums of exps are compared without the total that all share
    Pair total = {1.0f, 0.0f};
    if (!p.sigmoid && p.bias) total = total_pair(p, row, lane, L, k.m);
    uint64_t c[kMaxPerLane];
    uint32_t known = first_keys(p, row, a, k, bias, scored, total.hi, c);
#pragma unroll 1
    for (;;) {
        uint64_t g1 = 0u, g2 = 0u;
#pragma unroll 1
        for (int i = 0; i < a.n; ++i) best_two(g1, g2, c[i], (uint64_t)0u);
#pragma unroll 1
        for (int o = (1 << p.lane_shift) / 2; o; o >>= 1) {
            const uint64_t b1 = shfl_xor_key(g1, o), b2 = shfl_xor_key(g2, o);
            best_two(g1, g2, b1, b2);
        }
        const bool two = sums && g2 != 0u;
        const uint64_t v = sums ? half_sum_key(g1, g2) : g1;
        int rank = 0;
        float edge = 0.0f, next = 0.0f;  // the last value that is chosen, the first that is not
#pragma unroll 1
        for (int h = 0; h < p.groups; ++h) {
            const uint64_t u = __shfl_sync(kAll, (unsigned long long)v, h << p.lane_shift, L);
            rank += u > v || (u == v && h < a.group);
        }
#pragma unroll 1
        for (int h = 0; h < p.groups; ++h) {
            const float u = __shfl_sync(kAll, key_hi(v), h << p.lane_shift, L);
            const int r = __shfl_sync(kAll, rank, h << p.lane_shift, L);
            if (r == p.topk_groups - 1) edge = u;
            if (r == p.topk_groups) next = u;
        }
        const float low = key_hi(two ? g2 : g1), value = key_hi(v);
        const float part = sums ? 0.5f : 1.0f;
        const float size =
            __fadd_rn(fabsf(part * key_hi(g1)), two ? fabsf(part * low) : 0.0f);
        const float near = __fmaf_rn(1e-6f, size, 2.0f * k.tol);
        const bool open = scored && g1 != 0u && p.topk_groups < p.groups &&
                          (rank < p.topk_groups ? value - next <= near : edge - value <= near);
        const float from = __fmaf_rn(-1e-6f, fabsf(low), low - k.tol);
        bool more = false;
#pragma unroll 1
        for (int i = 0; open && i < a.n; ++i)
            if (!((known >> i) & 1u) && c[i] != 0u && key_hi(c[i]) >= from) {
                c[i] = value_key(p.sigmoid, load_any(row, a.j0 + i, p.dt),
                                 bias ? __ldg(p.bias + a.j0 + i) : 0.0f, k.m, total);
                known |= 1u << i;
                more = true;
            }
        if (!__any_sync(kAll, more)) return rank < p.topk_groups;
    }
}

// The border between two groups, the last that is chosen (side 1) and the first that is
// not (side 2), where no third is near: whether the second comes first.  The lanes of the
// two know, by bits of `terms`, which of their values can be among those that count.
__device__ __noinline__ bool swap_groups(const ScoredParams &p, const uint8_t *row, int lane, int L,
                                         Token k, int side, uint32_t terms, int one, int other) {
    constexpr unsigned kAll = 0xFFFFFFFFu;
    const Place a = place_of(p, lane % L);
    const bool bias = p.bias && !k.plain;
    Pair total = {1.0f, 0.0f};
    if (!p.sigmoid && p.bias) total = total_pair(p, row, lane, L, k.m);
    uint64_t g1 = 0u, g2 = 0u;
#pragma unroll 1
    for (uint32_t todo = side ? terms : 0u; todo; todo &= todo - 1) {
        const int j = a.j0 + __ffs((int)todo) - 1;
        const uint64_t c = value_key(p.sigmoid, load_any(row, j, p.dt),
                                     bias ? __ldg(p.bias + j) : 0.0f, k.m, total);
        best_two(g1, g2, c, (uint64_t)0u);
    }
#pragma unroll 1
    for (int o = (1 << p.lane_shift) / 2; o; o >>= 1) {
        const uint64_t b1 = shfl_xor_key(g1, o), b2 = shfl_xor_key(g2, o);
        best_two(g1, g2, b1, b2);
    }
    if (p.top2) g1 = half_sum_key(g1, g2);
    const uint64_t u = __shfl_sync(kAll, (unsigned long long)g1, one, L);
    const uint64_t v = __shfl_sync(kAll, (unsigned long long)g1, other, L);
    return v > u || (v == u && other < one);
}

// The choice from all of a token's values, for a warp with one that the kept keys do not
// decide; lane r of each token gets choice r (-1: none left).  in: whether the lane's
// group is chosen.  Values in fp32, those near the one that is chosen as pairs too.
__device__ __noinline__ int choose_again(const ScoredParams &p, const uint8_t *row, int lane, int L,
                                         bool in, Token k) {
    constexpr unsigned kAll = 0xFFFFFFFFu;
    const int sub = lane % L;
    const Place a = place_of(p, sub);
    const bool bias = p.bias && !k.plain;
    Pair total = {1.0f, 0.0f};
    if (!p.sigmoid && p.bias) total = total_pair(p, row, lane, L, k.m);
    uint64_t c[kMaxPerLane];
    uint32_t known = first_keys(p, row, a, k, bias, bias, total.hi, c);
    int id = -1;
#pragma unroll 1
    for (int r = 0; r < p.top_k; ++r) {
        uint64_t best;
        int at;
#pragma unroll 1
        for (;;) {
            best = 0u;
            at = 0x7FFFFFFF;
#pragma unroll 1
            for (int i = 0; in && i < a.n; ++i)
                if (c[i] > best) {
                    best = c[i];
                    at = a.j0 + i;
                }
#pragma unroll 1
            for (int o = L / 2; o; o >>= 1) {
                const uint64_t v = shfl_xor_key(best, o);
                const int j = __shfl_xor_sync(kAll, at, o);
                if (v > best || (v == best && j < at)) {
                    best = v;
                    at = j;
                }
            }
            const float hi = key_hi(best);
            const float from = __fmaf_rn(-1e-6f, fabsf(hi), hi - k.tol);
            uint32_t todo = 0u;
            int count = 0;
#pragma unroll 1
            for (int i = 0; bias && in && i < a.n; ++i)
                if (c[i] != 0u && key_hi(c[i]) >= from) {
                    ++count;
                    todo |= 1u << i;
                }
#pragma unroll 1
            for (int o = L / 2; o; o >>= 1) count += __shfl_xor_sync(kAll, count, o);
            todo = count > 1 ? todo & ~known : 0u;
            if (!__any_sync(kAll, todo != 0u)) break;
            known |= todo;
#pragma unroll 1
            for (; todo; todo &= todo - 1) {
                const int i = __ffs((int)todo) - 1;
                c[i] = value_key(p.sigmoid, load_any(row, a.j0 + i, p.dt), __ldg(p.bias + a.j0 + i),
                                 k.m, total);
            }
        }
        if (in && at >= a.j0 && at < a.j0 + a.n) c[at - a.j0] = 0u;
        if (sub == r) id = best != 0u ? at : -1;
    }
    return id;
}

// A row's 16-byte pieces lie in shared memory by the lane that they belong to, C for
// each, so that the lanes' reads of one after another, 8 at a time, meet all banks.
template <int C>
__device__ __forceinline__ int piece_at(int owner, int i) {
    static_assert(C >= 1 && C <= 8 && (C & (C - 1)) == 0, "pieces of a lane");
    return owner * C + (i ^ ((owner / (8 / C)) & (C - 1)));
}

// load_row where the lanes' logits are the whole row, in order: read as the row lies,
// lane after lane, and handed over.  (Each lane reading its own meets a line in each
// lane: 65537 x 256 forward 49 us, 38 this way.)
template <int DT, int NV, int L>
__device__ __forceinline__ void load_row_staged(const uint8_t *row, int lane, uint4 *warp_buf,
                                                float (&x)[NV]) {
    constexpr int C = NV * kSize<DT> / 16, W = 16 / kSize<DT>;
    const int sub = lane % L;
    uint4 *buf = warp_buf + lane / L * (L * C);
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int at = k * L + sub;
        buf[piece_at<C>(at / C, at % C)] = __ldg(reinterpret_cast<const uint4 *>(row) + at);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const uint4 u = buf[piece_at<C>(sub, i)];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < W; ++j)
            x[i * W + j] = logit_of<DT>(DT == MOEQ_FP32 ? w[j * kSize<DT> / 4]
                                                        : (w[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
    }
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


template <int NV, int L, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(kWarps * 32) gate_scored_kernel(ScoredParams p) {
    constexpr unsigned kAll = 0xFFFFFFFFu;
    constexpr uint32_t kIdx = (uint32_t)(L * NV) - 1u;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane % L;
    const int64_t slot =
        ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * (32 / L) + lane / L;
    const bool active = slot < p.num_tokens;
    const int64_t t = active ? slot : p.num_tokens - 1;
    const uint8_t *row = p.logits + t * p.stride;
    const Place a = place_of(p, sub);
    // (16-bit logits of 8 a lane are a piece each)
    constexpr bool kStaged = L < 32 && NV >= 8;
    __shared__ uint4 rows_buf[kStaged ? kWarps * 32 * NV / 4 : 1];
    __shared__ uint4 bias_buf[kStaged && BIAS ? L * NV / 4 : 1];
    float x[NV];
    if (kStaged && p.staged && (p.dt == MOEQ_FP32 || NV > 8)) {
        uint4 *buf = rows_buf + (kStaged ? (threadIdx.x >> 5) * (32 * NV / 4) : 0);
        if constexpr (kStaged) {
            if (p.dt == MOEQ_FP32) {
                load_row_staged<MOEQ_FP32, NV, L>(row, lane, buf, x);
            } else if constexpr (NV > 8) {
                if (p.dt == MOEQ_BF16)
                    load_row_staged<MOEQ_BF16, NV, L>(row, lane, buf, x);
                else
                    load_row_staged<MOEQ_FP16, NV, L>(row, lane, buf, x);
            }
        }
    } else if (p.dt == MOEQ_FP32)
        load_row<MOEQ_FP32>(row, a.j0 + a.n, a.j0, p.vec, x);
    else if (p.dt == MOEQ_BF16)
        load_row<MOEQ_BF16>(row, a.j0 + a.n, a.j0, p.vec, x);
    else
        load_row<MOEQ_FP16>(row, a.j0 + a.n, a.j0, p.vec, x);
    bool usable = true;
#pragma unroll
    for (int i = 0; i < NV; ++i) usable &= x[i] > -kInf;
    float m = -kInf, total = 0.0f, inv = 0.0f;
    bool plain = false;  // no softmax: by the logits
    float e[NV];
    if constexpr (!SIGMOID) {
#pragma unroll
        for (int i = 0; i < NV; ++i) m = fmaxf(m, x[i]);
        m = lanes_top<L>(m);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            e[i] = exp_fast(x[i], m);
            total = __fadd_rn(total, e[i]);
        }
        total = lanes_sum<L>(total);
        if (!(m > -kInf)) total = 0.0f;
        inv = rcp_fast(total);
        plain = !(total < kInf);  // NaN: a NaN logit, or m infinite
    }
    // c, -inf for what is never chosen
    auto value = [&](float v, float b) {
        if constexpr (!BIAS) return v;
        if constexpr (SIGMOID) return __fadd_rn(score_fast(v), b);
        return plain ? v : __fadd_rn(__fmul_rn(exp_fast(v, m), inv), b);
    };
    float c[NV];
    if constexpr (BIAS) {
        if (kStaged && p.staged) {
            constexpr int C = kStaged ? NV / 4 : 1;
            for (int at = threadIdx.x; at < L * C; at += kWarps * 32)
                bias_buf[piece_at<C>(at / C, at % C)] =
                    __ldg(reinterpret_cast<const uint4 *>(p.bias) + at);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const uint4 u = bias_buf[piece_at<C>(sub, i)];
                c[(4 * i) % NV] = __uint_as_float(u.x);
                c[(4 * i + 1) % NV] = __uint_as_float(u.y);
                c[(4 * i + 2) % NV] = __uint_as_float(u.z);
                c[(4 * i + 3) % NV] = __uint_as_float(u.w);
            }
        } else if (p.bias_vec && a.n == NV) {
#pragma unroll
            for (int i = 0; i < NV; i += 4) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(p.bias + a.j0 + i));
                c[i] = u.x;
                if (i + 3 < NV) {
                    c[(i + 1) % NV] = u.y;
                    c[(i + 2) % NV] = u.z;
                    c[(i + 3) % NV] = u.w;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) c[i] = i < a.n ? __ldg(p.bias + a.j0 + i) : 0.0f;
        }
        // a NaN as -inf
        if constexpr (SIGMOID) {
#pragma unroll
            for (int i = 0; i < NV; ++i) c[i] = fmaxf(value(x[i], c[i]), -kInf);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                c[i] = fmaxf(plain ? x[i] : __fadd_rn(__fmul_rn(e[i], inv), c[i]), -kInf);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = x[i];
    }
    bool nan = false;
    if (__any_sync(kAll, !usable)) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            nan |= x[i] != x[i];
            c[i] = x[i] > -kInf ? c[i] : -kInf;
        }
    }
    // How far apart two values are decided: twice the scores' bound, and the rounding of
    // the sums with the bias (2^-24 each, taken as 2^-22).
    const float tol = SIGMOID ? 2.0f * kScoreTol : 2.0f * kSoftmaxTol * inv;
    const bool rounded = BIAS && !plain;
    bool in = true;  // the lane's group is chosen
    if (p.groups > 1) {
        const bool sum = p.top2 && !plain, scores = sum && !BIAS;
        float g1 = -kInf, g2 = -kInf;
        if (scores) {  // exp without the total, which all share
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float v = SIGMOID ? score_fast(c[i]) : e[SIGMOID ? 0 : i];
                best_two(g1, g2, c[i] > -kInf ? v : -kInf, -kInf);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                g2 = fmaxf(g2, fminf(g1, c[i]));
                g1 = fmaxf(g1, c[i]);
            }
        }
        for (int o = (1 << p.lane_shift) / 2; o; o >>= 1) {
            const float b1 = __shfl_xor_sync(kAll, g1, o), b2 = __shfl_xor_sync(kAll, g2, o);
            best_two(g1, g2, b1, b2);
        }
        const bool two = sum && g2 > -kInf;
        // of sums their halves: that of two biases of the type's lowest value is not in fp32
        const float part = sum ? 0.5f : 1.0f;
        const float v = __fadd_rn(part * g1, two ? part * g2 : 0.0f);
        // groups by their values' images, the lowest of equal ones first
        uint32_t key = a.group < p.groups ? order_key(v) : 0u, border = 0u;
        int at = 0;  // the first lane of the group chosen last
        in = false;
        for (int r = 0; r < p.topk_groups; ++r) {
            border = lanes_max<L>(key);
            const uint32_t has = __ballot_sync(kAll, key == border) >> (lane - sub);
            at = __ffs((int)has) - 1;
            if (a.group == at >> p.lane_shift) {
                in = true;
                key = 0u;
            }
        }
        // (the tokens of a warp may differ in plain: what is between lanes runs for all)
        if (p.topk_groups < p.groups && (p.top2 || BIAS)) {
            // The border between the last group chosen and the first that is not.  A group
            // whose distance from the far side of it is within twice its own error is
            // not decided.  (Of a chosen and another one in the wrong order, one at least is
            // that: they lie no further apart than their two errors, and each no further
            // from the border.  Values that cancel have a larger error than their neighbours.)
            const uint32_t next = lanes_max<L>(key);
            const float bound = BIAS || SIGMOID ? tol : 2.0f * kExpTol;
            const float size = __fadd_rn(fabsf(part * g1), two ? fabsf(part * g2) : 0.0f);
            const float error = v < kInf ? __fmaf_rn(size, 0x1p-21f, part * bound) : 0.0f;
            const float vb = key_value(border), vn = key_value(next);
            const float gap = __fadd_rn(in ? v : vb, in ? -vn : -v);
            const uint32_t undecided = __ballot_sync(
                kAll, (sum || rounded) && next > kNegInfKey && v > -kInf && !(gap > 2.0f * error));
            if (undecided) {
                const bool unsure = ((undecided >> (lane - sub)) & (kAll >> (32 - L))) != 0u;
                const uint32_t has = __ballot_sync(kAll, key == next) >> (lane - sub);
                const int other = __ffs((int)has) - 1;
                // a third one as near, from either side
                const int side = a.group == at >> p.lane_shift      ? 1
                                 : a.group == other >> p.lane_shift ? 2
                                                                    : 0;
                const float most =
                    fmaxf(__shfl_sync(kAll, error, at, L), __shfl_sync(kAll, error, other, L));
                const float wide = 2.0f * __fadd_rn(error, most);
                const bool third = unsure && (side == 0 ? v > -kInf && !(gap > wide)
                                                        : !(size < 1e30f));
                const Token token{m, plain, bound};
                if (__any_sync(kAll, third)) {
                    in = groups_again(p, row, lane, L, token);
                } else {
                    uint32_t terms = 0u;
                    const float low = two ? g2 : g1;
                    const float from = __fadd_rn(low, -__fmaf_rn(fabsf(low), 0x1p-20f, bound));
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const float u = scores ? (SIGMOID ? score_fast(c[i]) : e[SIGMOID ? 0 : i])
                                               : c[i];
                        if (c[i] > -kInf && u >= from) terms |= 1u << i;
                    }
                    if (!unsure) terms = 0u;
                    const bool swap = swap_groups(p, row, lane, L, token, side, terms, at, other);
                    if (unsure && swap) in = side == 1 ? false : side == 2 ? true : in;
                }
            }
        }
    }
    float top = -kInf;
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, c[i]);
    top = lanes_top<L>(in ? top : -kInf);
    // without a bias the images of 16-bit logits are whole in the bits above the index
    const bool whole = !BIAS && p.dt != MOEQ_FP32;
    // keys from that of -inf, or of an infinite distance, on stand for no expert
    const uint32_t none = whole ? ~kNegInfKey >> 1 : 0x7F800000u;
    // half the distance, which cannot overflow
    const float half = __fmul_rn(top, 0.5f);
    uint32_t key[NV];
    if (whole) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = ~order_key(c[i]) >> 1;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            key[i] = __float_as_uint(__fmaf_rn(c[i], -0.5f, half)) & 0x7FFFFFFFu;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = (key[i] & ~kIdx) | (uint32_t)(sub * NV + i);
    // a token's best keys, and the one behind them; of a lane's at most as many as that
    // (top_k <= L) and one are looked at
    constexpr int kKeep = NV < L + 2 ? NV : L + 2;
    constexpr uint32_t kNoKey = 0x7FFFFFFFu;
    __shared__ uint32_t chosen[kWarps][32 / L][L + 1];
    uint32_t *out = chosen[threadIdx.x >> 5][lane / L];
    if (L < 32 && NV >= 16 && p.halves) {
        // a lane is a group, and no more than half of them are chosen: each other lane
        // sorts the second half of a chosen one's keys (65537 x 256 forward 38 us, 36)
        constexpr int H = NV > 1 ? NV / 2 : 1;
        constexpr uint32_t kLanes = L < 32 ? (1u << (L % 32)) - 1u : kAll;
        const uint32_t ins = (__ballot_sync(kAll, in) >> (lane - sub)) & kLanes;
        const int rank = __popc((in ? ins : ~ins) & ((1u << sub) - 1u));
        if (in) out[rank] = (uint32_t)sub;
        __syncwarp();
        const bool takes = !in && rank < __popc(ins);
        const int from = takes ? (int)out[rank] : sub;
        __syncwarp();
        uint32_t half_keys[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const uint32_t u = __shfl_sync(kAll, key[(H + i) % NV], from, L);
            half_keys[i] = in ? key[i] : takes ? u : kNoKey;
        }
        merge_step<H, 1, 1>(half_keys);
#pragma unroll
        for (int i = 0; i < kKeep; ++i) key[i] = i < H ? half_keys[i % H] : kNoKey;
    } else {
        merge_step<NV, 1, 1>(key);
        if (p.groups > 1) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i) key[i] = in ? key[i] : kNoKey;
        }
    }
    for (int r = 0; r <= p.top_k; ++r) {
        const uint32_t mn = lanes_min<L>(key[0]);
        const bool own = key[0] == mn;
        if (own) out[r] = mn;
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            key[i] = own ? (i + 1 < kKeep ? key[(i + 1) % NV] : kNoKey) : key[i];
    }
    __syncwarp();
    auto expert_of = [&](uint32_t k) {
        const Place b = place_of(p, (int)((k & kIdx) / NV));
        return b.j0 + (int)(k & kIdx) % NV;
    };
    uint32_t rest = lanes_min<L>(key[0]);  // the best key that is left
    int id = -1;
    float v = 0.0f, b = 0.0f, cv = -kInf;
    auto candidate = [&]() {
        if (out[sub] < none) {
            id = expert_of(out[sub]);
            v = load_any(row, id, p.dt);
            if (BIAS) b = __ldg(p.bias + id);
            cv = value(v, b);
        }
    };
    // with a choice in each lane all have the one behind them beside their own
    const bool full = p.top_k == L;
    const int behind = full && out[L] < none ? expert_of(out[L]) : -1;
    float v_behind = 0.0f, b_behind = 0.0f;
    if (behind >= 0) {
        v_behind = load_any(row, behind, p.dt);
        if (BIAS) b_behind = __ldg(p.bias + behind);
    }
    if (sub <= p.top_k) candidate();
    // two neighbours that are not decided (of the same logit and bias the lower index
    // is first); lane top_k has the one behind the choices
    float vn = __shfl_down_sync(kAll, v, 1, L), bn = __shfl_down_sync(kAll, b, 1, L);
    float cn = __shfl_down_sync(kAll, cv, 1, L);
    if (full && sub == L - 1) {
        vn = v_behind;
        bn = b_behind;
        cn = behind >= 0 ? value(vn, bn) : -kInf;
    }
    const float near =
        rounded ? __fadd_rn(tol, __fmul_rn(fmaxf(fabsf(cv), fabsf(cn)), 0x1p-22f)) : 0.0f;
    bool unsure = !whole && sub < p.top_k && cn > -kInf && (v != vn || b != bn) &&
                  !(__fadd_rn(cv, -cn) > near);
    // whether what is left may be as good as the lane's choice: a bound of it is known (an
    // index took the key's low bits, so that the last choice need not be the lowest one)
    auto open = [&](uint32_t left) {
        const float bound = __fadd_rn(top, -2.0f * __uint_as_float(left & ~kIdx));
        const float slack = __fmul_rn(__fadd_rn(fabsf(top), fabsf(bound)), 0x1p-22f);
        return !whole && sub < p.top_k && id >= 0 && left < none &&
               !(__fadd_rn(cv, -bound) > __fadd_rn(near, slack));
    };
    bool all = !whole && top == kInf;
    unsure |= open(rest);
    const Token token{m, plain, tol};
    if (__any_sync(kAll, unsure | all)) {
        // more candidates, as many as there are lanes
        int count = full ? L : p.top_k + 1;
        if (__any_sync(kAll, open(rest))) {
#pragma unroll 1
            for (; count < L; ++count) {
                const uint32_t mn = lanes_min<L>(key[0]);
                const bool own = key[0] == mn;
                if (own) out[count] = mn;
#pragma unroll
                for (int i = 0; i < kKeep; ++i)
                    key[i] = own ? (i + 1 < kKeep ? key[(i + 1) % NV] : kNoKey) : key[i];
            }
            __syncwarp();
            if (sub > p.top_k) candidate();
            rest = lanes_min<L>(key[0]);
            all |= open(rest);
        }
        if (__any_sync(kAll, all)) {
            id = choose_again(p, row, lane, L, in, token);
        } else {
            // the candidates by their values as pairs; with a choice in each lane the one
            // behind them too, which every lane has
            uint64_t key64 = float_key(v), last = 0u;
            if (behind >= 0) last = float_key(v_behind);
            if (BIAS) {
                Pair sum = {1.0f, 0.0f};
                if (!SIGMOID) sum = total_pair(p, row, lane, L, m);
                if (!plain) {
                    key64 = value_key(SIGMOID, v, b, m, sum);
                    if (behind >= 0) last = value_key(SIGMOID, v_behind, b_behind, m, sum);
                }
            }
            int rank = behind >= 0 && (last > key64 || (last == key64 && behind < id));
            int place = 0;  // of the one behind
#pragma unroll 1
            for (int r = 0; r < count; ++r) {
                const uint64_t u = __shfl_sync(kAll, (unsigned long long)key64, r, L);
                const int j = __shfl_sync(kAll, id, r, L);
                rank += j >= 0 && (u > key64 || (u == key64 && j < id));
                place += j >= 0 && (u > last || (u == last && j < behind));
            }
            __syncwarp();
            out[sub] = 0xFFFFFFFFu;
            __syncwarp();
            if (id >= 0) out[rank] = (uint32_t)id;
            if (behind >= 0 && sub == 0) out[place] = (uint32_t)behind;
            __syncwarp();
            id = (int)out[sub];
        }
        if (sub < p.top_k && id >= 0) v = load_any(row, id, p.dt);
    }
    if (sub >= p.top_k) id = -1;
    // the weights
    const bool some = __shfl_sync(kAll, id, 0, L) >= 0;
    float s = 0.0f, sum = 0.0f;
    if (SIGMOID) {
        if (id >= 0) s = sigmoid_exact(v);
        sum = p.normalize ? s : 1.0f;
    } else if (p.normalize) {
        // relative to the largest of the chosen
        const float mc = lanes_top<L>(id >= 0 && v == v ? v : -kInf);
        if (id >= 0) s = exp_diff(v, mc);
        sum = s;
    } else {
        if (id >= 0) s = exp_diff(v, m);
        sum = total;
    }
    if (p.normalize) sum = lanes_sum<L>(sum);
    float w = sum > 0.0f ? __fmul_rn(__fdiv_rn(s, sum), p.scale) : 0.0f;
    // a NaN, or an infinity in a softmax, is seen in all of the token's weights
    const uint32_t nans = __ballot_sync(kAll, nan);
    if (plain || ((nans >> (lane - sub)) & (kAll >> (32 - L))) != 0u)
        w = __int_as_float(0x7FFFFFFF);
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
    // the zeros leave while the ids are on their way
    int id = -1;
    float g = 0.0f, x = -kInf;
    if (sub < p.top_k) {
        id = __ldg(p.ids + t * p.top_k + sub);
        g = __ldg(p.d_weights + t * p.top_k + sub);
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
    if (id < -1 || id >= p.E) {
        if (active) set_error(p.err, MOEQ_DEVERR_BAD_EXPERT);
        id = -1;
    }
    g = id >= 0 ? __fmul_rn(g, p.scale) : 0.0f;
    if (id >= 0) x = load_logit<DT>(in, id);
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

template <int NV, int L>
cudaError_t run_lanes(const ScoredParams &p, cudaStream_t s) {
    const int64_t per_cta = kWarps * 32 / L;
    auto *kern = p.sigmoid ? (p.bias ? gate_scored_kernel<NV, L, true, true>
                                     : gate_scored_kernel<NV, L, true, false>)
                           : (p.bias ? gate_scored_kernel<NV, L, false, true>
                                     : gate_scored_kernel<NV, L, false, false>);
    return launch_pdl(kern, (unsigned)((p.num_tokens + per_cta - 1) / per_cta), kWarps * 32, 0, s,
                      p);
}

// The lanes and logits per lane of a token's groups on L lanes, and the registers that
// a lane needs for them (a power of two); 0 where they do not fit.
int lay_out(ScoredParams &p, int L) {
    const int size = p.dt == MOEQ_FP32 ? 4 : 2;
    int lanes = L;  // of a group
    while (lanes > 0 && lanes * p.groups > L) lanes /= 2;
    if (lanes == 0 || p.top_k > L) return 0;
    p.group_size = p.E / p.groups;
    p.per_lane = (p.group_size + lanes - 1) / lanes;
    if (p.per_lane > kMaxPerLane) return 0;
    p.lane_shift = 0;
    while ((1 << p.lane_shift) < lanes) ++p.lane_shift;
    int nv = 1;
    while (nv < p.per_lane) nv *= 2;
    if (p.groups == 1) p.per_lane = nv;  // whole vectors
    const int bytes = std::min(nv * size, 16);
    const bool whole = p.per_lane == nv;  // lanes begin at multiples of nv in their group
    p.vec = whole && p.stride % bytes == 0 && (p.groups == 1 || p.group_size * size % bytes == 0);
    p.bias_vec = whole && nv % 4 == 0 && (p.groups == 1 || p.group_size % 4 == 0);
    p.halves = p.groups == L && 2 * p.topk_groups <= L;
    p.staged = p.vec && p.E == L * nv && (p.groups << p.lane_shift) == L;
    return nv;
}

cudaError_t run_scored(ScoredParams p, cudaStream_t s) {
    // Many tokens: few lanes each, so that what a token costs whatever its experts is
    // shared by the tokens of a warp.  Forward, sigmoid with bias, bf16, 8 lanes (or 16)
    // against 32: 65536 tokens x 64 experts, top-8, 17.7 / 37.8 us, x 128, top-4, 18.0 /
    // 35.7, x 160, 8 groups, 33.8 / 55.3, x 256, 8 groups, 33.4 (46.0) / 51.5, x 512, 16
    // groups (88) / 79; 4096 x 64 3.8 / 4.9, x 128 4.9 / 4.8, x 256 7.3 / 6.7
    ScoredParams q = p;
    if (p.num_tokens >= 4096) {
        const int nv = lay_out(q, 8);
        if (nv == 32) return run_lanes<32, 8>(q, s);
        if (nv == 16) return run_lanes<16, 8>(q, s);
        if (nv == 8) return run_lanes<8, 8>(q, s);
        if (nv == 4) return run_lanes<4, 8>(q, s);
    }
    if (p.num_tokens >= 8192) {
        const int nv = lay_out(q, 16);
        if (nv == 16) return run_lanes<16, 16>(q, s);
        if (nv == 8) return run_lanes<8, 16>(q, s);
    }
    const int nv = lay_out(p, 32);
    return nv == 0    ? cudaErrorNotSupported
           : nv == 1  ? run_lanes<1, 32>(p, s)
           : nv == 2  ? run_lanes<2, 32>(p, s)
           : nv == 4  ? run_lanes<4, 32>(p, s)
           : nv == 8  ? run_lanes<8, 32>(p, s)
           : nv == 16 ? run_lanes<16, 32>(p, s)
                      : run_lanes<32, 32>(p, s);
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
    p.dt = a.dtype;
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
    return run_scored(p, s);
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
