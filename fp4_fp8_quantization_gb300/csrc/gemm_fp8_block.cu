// Grouped FP8 GEMM with a scale for each block of 128 of the reduction:
//
//   c[t, n] = bf16( sum_kb (sa[t, kb] sb[e, n / 128, kb]) P_kb[t, n] ),
//   P_kb[t, n] = sum over k in block kb of a[t, k] b[e, n, k]
//
// The tensor cores can only apply power-of-two block scales, so P_kb (fp32,
// in tensor memory) is scaled outside: the warps that would be an epilogue
// run along the whole reduction.  Per K block of 128, one 128-byte swizzle
// row per operand row:
//  * warp 0 (one thread) loads the A and B tiles by TMA into a ring of
//    stages (columns past K and rows past N arrive as zeros);
//  * warp 1 (one thread) issues the block's four MMAs into one of NBUF
//    tensor-memory accumulators, overwriting it;
//  * the other warps read it (one row per thread, COLS_W columns per warp)
//    and add it, times the row's and column block's scales, to sums that stay
//    in registers for the whole tile.  A warp's columns lie in one 128-column
//    block, so the factor is one number per thread and K block: the pass is
//    one paired fused multiply-add per two elements.
// Persistent CTAs, one per SM, walk the tiles of all groups (n fastest).
// Every wait is bounded and sets the device error word instead of hanging.
//
// What bounds it: with many rows, about 700 cycles of a K block (128 x 256 tile)
// whose MMAs take 512.  Two things lie just above them: 48 KB of operands come
// into the SM (70 bytes a cycle; more requests or reads of them slow it at once,
// below), and the two accumulators' chain of MMAs, commit, 560 cycles of loads
// and sums, and release.  Above that is the power limit: 65536 x 7168 x 4096,
// 64 experts, 1.43 to 1.54 ms a single launch (2.7 to 2.5 PFLOP/s), 1.62 to 1.72
// back to back at about 1.5 GHz (2.4 to 2.2); the rowwise-scaled GEMM on the same
// operands 1.33 and 1.54.
// With few rows the stream of the weights: 512 rows over 256 experts, K 7168, N
// 4096, 0.93 ms, 103 % of the copy rate.  With sizes that end inside tiles
// (11996 rows over 48 experts, K 2480, N 1880: 99 us, 44 of memory), the whole
// tiles that a group's last rows and the last columns cost (the MMA's N and the
// weights' box are a tile's, 2048 columns for 1880), rows that start inside lines
// (K 2560: 74), and seven waves for 6.2 of tiles dealt out by number.
// What did not help: 64-column tensor-memory loads, polling waits, a second
// issuing warp (all within 1 %), the scales brought to shared memory by the two
// idle warps (10 % slower: the wait for them joins each block's chain), CTAs of
// 128 x 128 (30 %), an accumulator handed over by halves of 128 columns (10 %: A
// is read twice), 16 sum warps of 64 columns (11 %), MMAs over CTA pairs (7 %:
// each block waits for the sums of both), prefetches into L2 (10 %, 40 % for
// rows that start inside lines: the load path has no requests to spare).  In the
// small tile the weights as the MMAs' rows and the rows as their columns, which
// wastes no MMA rows, 4 % faster to 12 % slower (512 rows, 8 experts): the stream
// is what bounds it.  The reduction split over a cluster whose CTAs exchange their
// sums costs 2 us a tile: 24 tiles of K 4096 10.5 -> 8.1 us, 48 11.2 -> 10.7, but
// 96 (one token, 8 experts, N 1536) 13.8 -> 18.8.
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "tensormap.h"

namespace moeq {

namespace {

template <int BM_, int BN_, int STAGES_, int SUM_WARPS_, bool ASYNC_, int KSUB_>
struct BlockCfg {
    static constexpr int MMA_M = 128;
    static constexpr int BM = BM_;     // rows of an m-block; the MMAs' other rows are dropped
    static constexpr int BN = BN_, STAGES = STAGES_, SUM_WARPS = SUM_WARPS_;
    static constexpr int BK = 128;
    static constexpr int KSUB = KSUB_;  // K blocks per stage, each with its accumulator
    static constexpr int ACC_COLS = KSUB * BN;
    static constexpr int NBUF = 512 / ACC_COLS < 4 ? 512 / ACC_COLS : 4;  // sets of accumulators
    static constexpr int TMEM_COLS = NBUF * ACC_COLS;
    static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;  // of one K block
    static constexpr int SUB_BYTES = A_BYTES + B_BYTES, STAGE_BYTES = KSUB * SUB_BYTES;
    static constexpr int COLS_W = BN / (SUM_WARPS / 4), CHUNKS_W = COLS_W / 32;
    static constexpr int SUM_WARP0 = 4;  // warps 0 and 1 work, 2 and 3 fill their warpgroup
    static constexpr int THREADS = 32 * (SUM_WARP0 + SUM_WARPS);
    // the sums and two 32-column loads do not fit the registers that all the
    // threads of an SM leave each: the control warpgroup gives up registers to
    // the sum warpgroups (setmaxnreg redistributes exactly the registers the
    // block is launched with; the host checks the compiled count before
    // launching)
    static constexpr int LAUNCH_REGS = 65536 / THREADS / 8 * 8;
    static constexpr bool NREG = COLS_W + 64 + 48 > LAUNCH_REGS;
    static constexpr int NREG_CTRL = COLS_W == 128 ? 56 : 80;
    static constexpr int NREG_SUM =
        NREG ? (THREADS * LAUNCH_REGS - 32 * SUM_WARP0 * NREG_CTRL) / (32 * SUM_WARPS) / 8 * 8 : 0;
    // staging per warp of its 32 rows: ASYNC all of its columns, which leave by
    // tensor stores during the next tile; else one 32-column chunk at a time
    static constexpr bool ASYNC = ASYNC_;
    static constexpr int BUF_BYTES = ASYNC ? 32 * COLS_W * 2 : 2048;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + SUM_WARPS * BUF_BYTES + 1024;
    static_assert(SMEM_BYTES + 12 * (kMaxGroups + 1) + 512 <= 227 * 1024, "shared memory per CTA");
    static_assert(!ASYNC || COLS_W % 64 == 0, "boxes of 64 columns");
    // an MMA reads MMA_M rows of A, past a smaller m-block's end whatever is there
    static_assert(B_BYTES + SUM_WARPS * BUF_BYTES >= (MMA_M - BM) * BK, "A reads stay inside");
    static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS <= 512, "tensor memory");
    // a stage's done barrier is not used again before its last use was summed
    static_assert(STAGES >= NBUF, "the sums tell apart two uses of a stage by parity");
    static_assert(STAGE_BYTES % 1024 == 0 && BM % 32 == 0, "stage alignment");
    static_assert(!NREG || (NREG_SUM >= LAUNCH_REGS && NREG_SUM <= 248 &&
                            32 * SUM_WARP0 * NREG_CTRL + 32 * SUM_WARPS * NREG_SUM <=
                                THREADS * LAUNCH_REGS),
                  "register split by warpgroups");
    static_assert(CHUNKS_W % 2 == 0, "the two load buffers alternate across K blocks");
    static_assert(COLS_W % 32 == 0 && 128 % COLS_W == 0, "a warp's columns share one scale");
};

struct BlockGemmParams {
    const uint32_t *offsets;
    const int32_t *expert_ids;
    int num_groups, num_experts;
    int64_t total_rows;
    int N, K;
    const float *a_scales, *b_scales;
    uint16_t *c;
    uint32_t *err;
};

// A value that every lane of the (converged) warp holds, in a form the
// compiler keeps in uniform registers.
__device__ __forceinline__ uint32_t warp_uniform(uint32_t v) {
    return __reduce_max_sync(0xFFFFFFFFu, v);
}

// Two fp32 -> two bf16 (round to nearest even), the first in the low half.
__device__ __forceinline__ uint32_t bf16x2(F2 v) {
    uint32_t b;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(f2_hi(v)), "f"(f2_lo(v)));
    return b;
}

// Waits for the thread's tensor-memory loads; r is written by them.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])::"memory");
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    gemm_fp8_block_kernel(const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmA32,
                          const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmC, const BlockGemmParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full_bar[C::STAGES], done_bar[C::STAGES], tempty_bar[C::NBUF];
    __shared__ uint64_t drain_bar;
    __shared__ uint32_t tmem_slot, stages_done;
    __shared__ int abort_flag;
    // per group: tiles before it, first row, expert
    __shared__ uint32_t prefix[kMaxGroups + 1];
    __shared__ int first_row[kMaxGroups + 1], expert[kMaxGroups];

    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = (int)warp_uniform(threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int G = p.num_groups;
    const int NB = (p.N + C::BN - 1) / C::BN;
    const int KB = (p.K + C::BK - 1) / C::BK;           // K blocks, and sets of KSUB
    const int KS = (KB + C::KSUB - 1) / C::KSUB;
    volatile int *abort_v = &abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&done_bar[s], 1);
        }
        for (int b = 0; b < C::NBUF; ++b) mbar_init(&tempty_bar[b], C::SUM_WARPS);
        mbar_init(&drain_bar, 1);
        abort_flag = 0;
        stages_done = 0;
        prefix[0] = 0;
        fence_barrier_init();
        if (C::BM == 128) prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmA32);
        prefetch_tensormap(&tmB);
    }
    // everything above touches only shared memory and the kernel parameters
    pdl_wait();
    if (warp == 1) {
        tmem_alloc(&tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    // tiles of each group; an unusable group has none and is reported once
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
        const uint32_t r0 = __ldg(p.offsets + g), r1 = __ldg(p.offsets + g + 1);
        const int e = __ldg(p.expert_ids + g);
        first_row[g] = (int)r0;
        if (g == G - 1) first_row[G] = (int)r1;
        expert[g] = e;
        uint32_t n = 0;
        if (r1 < r0 || (int64_t)r1 > p.total_rows) {
            if (blockIdx.x == 0) set_error(p.err, MOEQ_DEVERR_BAD_OFFSETS);
        } else if (e < 0 || e >= p.num_experts) {
            if (blockIdx.x == 0) set_error(p.err, MOEQ_DEVERR_BAD_EXPERT);
        } else {
            n = (r1 - r0 + C::BM - 1) / C::BM * (uint32_t)NB;
        }
        prefix[g + 1] = n;
    }
    __syncthreads();
    if (warp == 0) {  // inclusive prefix over prefix[1..G]
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t total = warp_uniform(prefix[G]);
    const uint32_t tmem = warp_uniform(tmem_slot);

    if (warp < C::SUM_WARP0) {
    if constexpr (C::NREG) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::NREG_CTRL));
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_last();
            int stage = 0;
            uint32_t phase = 0, issued = 0;
            bool ok = true;
            for (uint32_t t = blockIdx.x; ok && t < total; t += gridDim.x) {
                const Tile tl = decode_tile(prefix, G, t, NB);
                const int e = expert[tl.g], r1 = first_row[tl.g + 1];
                const int row0 = first_row[tl.g] + tl.mb * C::BM;
                // of a partial m-block only the 32-row boxes that hold rows of the
                // group are loaded; what the rest of the stage holds only reaches
                // rows that are dropped
                const int boxes = (min(r1 - row0, C::BM) + 31) / 32;
                const uint32_t tx = C::KSUB * (boxes * 32 * C::BK + C::B_BYTES);
                for (int kb = 0; kb < KS; ++kb) {
                    if (!mbar_wait(&done_bar[stage], phase ^ 1u, abort_v, p.err)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = smem + stage * C::STAGE_BYTES;
                    bool stuck = false;
#ifdef MOEQ_TEST_STUCK_STAGE
                    // failure-detection test build: the first stage of the CTA's
                    // first tile is announced but never loaded
                    stuck = t == blockIdx.x && kb == 0;
#endif
                    mbar_arrive_expect_tx(&full_bar[stage], tx);
                    ++issued;
                    if (stuck) {
                        if (++stage == C::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        continue;
                    }
#pragma unroll
                    for (int q = 0; q < C::KSUB; ++q) {  // past K: zeros
                        uint8_t *s = sa + q * C::SUB_BYTES;
                        const int k = (kb * C::KSUB + q) * C::BK;
                        if (C::BM == 128 && boxes == 4) {
                            tma_load_2d(s, &tmA, &full_bar[stage], k, row0, pol);
                        } else {
                            for (int i = 0; i < boxes; ++i)
                                tma_load_2d(s + i * 32 * C::BK, &tmA32, &full_bar[stage], k,
                                            row0 + i * 32, pol);
                        }
                        tma_load_3d(s + C::A_BYTES, &tmB, &full_bar[stage], k, tl.nb * C::BN, e, pol);
                    }
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            stages_done = issued;
        }
    } else if (warp == 1) {
        // the whole warp walks the loop (so that addresses and descriptors
        // are warp-uniform), one thread issues; one commit per K block tells
        // both the loads (stage free) and the sums (accumulator full)
        const bool leader = elect_one();
        const uint64_t da0 = sdesc_sw128(smem_u32(smem));
        const uint64_t db0 = sdesc_sw128(smem_u32(smem) + C::A_BYTES);
        int stage = 0, buf = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
        for (uint32_t t = blockIdx.x; ok && t < total; t += gridDim.x) {
            for (int kb = 0; kb < KS; ++kb) {
                // the operands are mostly there first: their wait is paid while
                // the accumulator is still being read
                ok = __all_sync(0xFFFFFFFFu,
                                mbar_wait(&full_bar[stage], phase, abort_v, p.err) &&
                                    mbar_wait(&tempty_bar[buf], bphase ^ 1u, abort_v, p.err));
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint32_t off = (uint32_t)(stage * C::STAGE_BYTES) >> 4;
#pragma unroll
                    for (int q = 0; q < 4 * C::KSUB; ++q) {
                        const uint32_t at = off + (q / 4) * (C::SUB_BYTES >> 4) + 2 * (q & 3);
                        mma_f8f6f4(tmem + buf * C::ACC_COLS + (q / 4) * C::BN, da0 + at, db0 + at,
                                   idesc_f8_e4m3(C::MMA_M, C::BN), q & 3 ? 1u : 0u);
                    }
                    tc_commit(&done_bar[stage]);
                }
                __syncwarp();
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++buf == C::NBUF) {
                    buf = 0;
                    bphase ^= 1u;
                }
            }
        }
        // every tcgen05 operation issued here completes before TMEM is freed
        if (leader) {
            tc_commit(&drain_bar);
            mbar_drain(&drain_bar, 0);
        }
        __syncwarp();
    }
    } else {
        if constexpr (C::NREG)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::NREG_SUM));
        const int quad = warp & 3;                    // TMEM lanes 32 quad .. 32 quad + 31
        const int cgrp = (warp - C::SUM_WARP0) >> 2;  // columns COLS_W cgrp ...
        const uint32_t toff = ((uint32_t)(quad * 32) << 16) + cgrp * C::COLS_W;
        const uint32_t sbuf = smem_u32(smem + C::STAGES * C::STAGE_BYTES) +
                              (warp - C::SUM_WARP0) * C::BUF_BYTES;
        const int NBLK = (p.N + 127) / 128;
        // what this warp has of a tile: rows [row, row + nvalid) and columns from
        // ncol, the scales of its lanes' rows and of its column block (a lane past
        // the last row takes that row's, its sums are dropped)
        struct Part {
            int row, nvalid, ncol;
            const float *sa, *sb;
            __device__ bool work(int N) const { return nvalid > 0 && ncol < N; }
        };
        auto part_of = [&](uint32_t t) {
            const Tile tl = decode_tile(prefix, G, t, NB);
            const int e = expert[tl.g], r1 = first_row[tl.g + 1];
            Part w;
            w.row = first_row[tl.g] + tl.mb * C::BM + quad * 32;
            w.nvalid = quad * 32 < C::BM ? max(0, min(32, r1 - w.row)) : 0;
            w.ncol = tl.nb * C::BN + cgrp * C::COLS_W;
            w.sa = p.a_scales + (int64_t)(w.row + max(0, min(lane, w.nvalid - 1))) * KB;
            w.sb = p.b_scales + ((int64_t)e * NBLK + min(w.ncol / 128, NBLK - 1)) * KB;
            return w;
        };
        // each lane polls by itself: where the barrier completes while another
        // warp gives up, some would go on and some leave, and what follows is the
        // whole warp's
        auto sums_wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_v, p.err));
        };
        int buf = 0, stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        Part cur = {}, nxt = {};
        // the scales of the next K block, on their way during this one
        float an[C::KSUB] = {}, bn[C::KSUB] = {};
        auto first_scales = [&]() {
#pragma unroll
            for (int q = 0; q < C::KSUB; ++q) {
                an[q] = nxt.work(p.N) && q < KB ? __ldg(nxt.sa + q) : 0.0f;
                bn[q] = nxt.work(p.N) && q < KB ? __ldg(nxt.sb + q) : 0.0f;
            }
        };
        if (blockIdx.x < total) {
            nxt = part_of(blockIdx.x);
            first_scales();
        }
        for (uint32_t t = blockIdx.x; ok && t < total; t += gridDim.x) {
            cur = nxt;
            const bool work = cur.work(p.N);
            F2 acc[C::COLS_W / 2];
#pragma unroll
            for (int i = 0; i < C::COLS_W / 2; ++i) acc[i] = f2(0.0f, 0.0f);
            if (!work) {  // only hands the accumulators on
                for (int kb = 0; kb < KS; ++kb) {
                    ok = sums_wait(&done_bar[stage], phase);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive(&tempty_bar[buf]);
                    if (++buf == C::NBUF) buf = 0;
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            } else {
            // the load of the next 32 columns (of the next K block at the end
            // of this one) is in flight while the last 32 are added
            uint32_t r[2][32];
            const float *sa = cur.sa, *sb = cur.sb;
            ok = sums_wait(&done_bar[stage], phase);
            if (!ok) break;
            tc_fence_after();
            tmem_ld32(tmem + buf * C::ACC_COLS + toff, r[0]);
            constexpr int CH = C::KSUB * C::CHUNKS_W;  // 32-column loads of a set
#pragma unroll 1
            for (int kb = 0; kb < KS; ++kb) {
                F2 s2[C::KSUB];
#pragma unroll
                for (int q = 0; q < C::KSUB; ++q) {
                    const float s = __fmul_rn(an[q], bn[q]);
                    s2[q] = f2(s, s);
                    const int k = (kb + 1) * C::KSUB + q;
                    if (k < KB) {
                        an[q] = __ldg(sa + k);
                        bn[q] = __ldg(sb + k);
                    } else if (C::KSUB > 1) {
                        an[q] = bn[q] = 0.0f;  // an absent block of the last set
                    }
                }
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    const int q = ch / C::CHUNKS_W, cc = ch % C::CHUNKS_W;
                    tmem_ld_wait32(r[ch & 1]);
                    if (ch < CH - 1) {
                        tmem_ld32(tmem + buf * C::ACC_COLS + toff +
                                      (ch + 1) / C::CHUNKS_W * C::BN + (ch + 1) % C::CHUNKS_W * 32,
                                  r[(ch + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tempty_bar[buf]);
                        if (++buf == C::NBUF) buf = 0;
                        if (++stage == C::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        if (kb + 1 < KS) {
                            // a warp that gives up leaves after the sums below,
                            // so that they do not wait for the vote
                            ok = sums_wait(&done_bar[stage], phase);
                            tc_fence_after();
                            tmem_ld32(tmem + buf * C::ACC_COLS + toff, r[0]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[cc * 16 + i] = fma2(f2(__uint_as_float(r[ch & 1][2 * i]),
                                                   __uint_as_float(r[ch & 1][2 * i + 1])),
                                                s2[q], acc[cc * 16 + i]);
                }
                if (!ok) {
                    tmem_ld_wait32(r[0]);
                    break;
                }
            }
            }
            if (!ok) break;
            // the next tile's place and first scales, while this one is stored
            if (t + gridDim.x < total) {
                nxt = part_of(t + gridDim.x);
                first_scales();
            }
            if (!work) continue;
            if constexpr (C::ASYNC) {
                // the whole part into the warp's staging buffer, in boxes of 64
                // columns (rows of 128 bytes in the tensor map's 128-byte swizzle);
                // the last tile's stores have long read it
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
#pragma unroll
                for (int ch = 0; ch < C::COLS_W / 64; ++ch)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const F2 *v = acc + ch * 32 + j * 4;
                        st_shared_v4(sbuf + ch * 4096 + lane * 128 + ((j ^ (lane & 7)) << 4),
                                     bf16x2(v[0]), bf16x2(v[1]), bf16x2(v[2]), bf16x2(v[3]));
                    }
                if (cur.nvalid == 32) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        // the box ends at N by its tensor map
                        for (int ch = 0; ch < C::COLS_W / 64; ++ch)
                            if (cur.ncol + ch * 64 < p.N &&
                                store_ok(cur.row >= 0 && cur.row + 32 <= p.total_rows, p.err))
                                tma_store_2d(&tmC, sbuf + ch * 4096, cur.ncol + ch * 64, cur.row);
                        bulk_commit();
                    }
                } else {  // the end of a group: its rows only, eight lanes each
                    __syncwarp();
                    const int k = lane & 7;
                    for (int ch = 0; ch < C::COLS_W / 64; ++ch) {
                        const int n = cur.ncol + ch * 64 + k * 8;
                        for (int rr = lane >> 3; rr < cur.nvalid; rr += 4) {
                            const uint4 v =
                                ld_shared_v4(sbuf + ch * 4096 + rr * 128 + ((k ^ (rr & 7)) << 4));
                            uint16_t *out = p.c + (int64_t)(cur.row + rr) * p.N + n;
                            if (n < p.N && store_fits(out, 16, p.c, p.total_rows * p.N * 2, p.err))
                                st_global_v4(out, v.x, v.y, v.z, v.w);
                        }
                    }
                }
                continue;
            }
            // bf16 out through the warp's 32 x 32 staging buffer (64-byte rows
            // whose 16-byte pieces are XOR-swizzled by row pair, free of bank
            // conflicts), stored with four lanes per row
            const int k = lane & 3, lrow = lane >> 2;
            uint16_t *out = p.c + (int64_t)(cur.row + lrow) * p.N + cur.ncol + k * 8;
#pragma unroll
            for (int ch = 0; ch < C::CHUNKS_W; ++ch) {
                const int nc = cur.ncol + ch * 32;
                if (nc >= p.N) break;
                __syncwarp();  // the last chunk has been read
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const F2 *v = acc + ch * 16 + j * 4;
                    st_shared_v4(sbuf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4), bf16x2(v[0]),
                                 bf16x2(v[1]), bf16x2(v[2]), bf16x2(v[3]));
                }
                __syncwarp();
                const bool in_n = nc + k * 8 < p.N;  // N is a multiple of 8
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rr = lrow + 8 * i;
                    const uint4 v = ld_shared_v4(sbuf + rr * 64 + ((k ^ ((rr >> 1) & 3)) << 4));
                    uint16_t *o = out + (int64_t)(8 * i) * p.N + ch * 32;
                    if (rr < cur.nvalid && in_n &&
                        store_fits(o, 16, p.c, p.total_rows * p.N * 2, p.err))
                        st_global_v4(o, v.x, v.y, v.z, v.w);
                }
            }
        }
        if (C::ASYNC && lane == 0) bulk_wait_all();
    }

    // this CTA's loads, MMAs and stores are all issued
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        // every issued copy lands before the CTA leaves, after an abort too
        const uint32_t v = stages_done;
        for (uint32_t s = 0; s < (uint32_t)C::STAGES; ++s) {
            const uint32_t n = v / C::STAGES + (s < v % C::STAGES ? 1u : 0u);
            if (n) mbar_drain(&full_bar[s], (n - 1) & 1u);
        }
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <class C>
cudaError_t run_block_gemm(const GemmBlockArgs &a, cudaStream_t s) {
    const int64_t T = a.groups.total_rows;
    // the whole-block map of A is of the 128-row tiles, the output's of the
    // asynchronous stores; a map takes the host about half a microsecond
    CUtensorMap tA = {}, tA32, tB, tC = {};
    cuuint64_t da[2] = {(cuuint64_t)a.K, (cuuint64_t)T};
    cuuint64_t sa[1] = {(cuuint64_t)a.K};
    cuuint64_t db[3] = {(cuuint64_t)a.K, (cuuint64_t)a.N, (cuuint64_t)a.groups.num_experts};
    cuuint64_t sb[2] = {(cuuint64_t)a.K, (cuuint64_t)(a.K * a.N)};
    // boxes of rows that start inside a 128-byte line: fetching 256 bytes for each
    // of them costs more than it brings (K 2608 99.7 us, 86.1 with 128 bytes; K
    // 2560 74.0 / 78.2; 12000 rows, N 1880, 48 experts)
    const CUtensorMapL2promotion promotion = a.K % 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                       : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    if ((C::BM == 128 && !make_map(&tA, a.a, 2, da, sa, 128, promotion)) ||
        !make_map(&tA32, a.a, 2, da, sa, 32, promotion) ||
        !make_map(&tB, a.b, 3, db, sb, C::BN, promotion))
        return cudaErrorInvalidValue;
    // bf16 output, boxes of 32 rows x 64 columns in the staging buffer's swizzle
    cuuint64_t dc[2] = {(cuuint64_t)a.N, (cuuint64_t)T};
    cuuint64_t sc[1] = {(cuuint64_t)a.N * 2};
    cuuint32_t bc[2] = {64, 32}, ec[2] = {1, 1};
    if (C::ASYNC &&
        encode_fn()(&tC, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.c, dc, sc, bc, ec,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_NONE,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const BlockGemmParams p{a.groups.row_offsets, a.groups.expert_ids, a.groups.num_groups,
                            a.groups.num_experts, T, (int)a.N, (int)a.K, a.a_scales, a.b_scales,
                            static_cast<uint16_t *>(a.c), a.err};
    auto kern = gemm_fp8_block_kernel<C>;
    static std::atomic<int> attr_done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    cudaError_t attr_err = cudaSuccess;
    cached_per_device(attr_done, dev, [&]() {
        attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        C::SMEM_BYTES);
        if (attr_err == cudaSuccess && C::NREG) {
            // the register split assumes THREADS x LAUNCH_REGS registers: refuse
            // to launch a build that differs
            cudaFuncAttributes fa;
            attr_err = cudaFuncGetAttributes(&fa, kern);
            if (attr_err == cudaSuccess && fa.numRegs < C::LAUNCH_REGS)
                attr_err = cudaErrorInvalidConfiguration;
        }
        return attr_err == cudaSuccess ? 1 : 0;
    });
    if (attr_err != cudaSuccess) return attr_err;
    // upper bound of the tiles the offsets can give
    const int64_t tiles = (T / C::BM + std::min<int64_t>(a.groups.num_groups, T)) *
                          ((a.N + C::BN - 1) / C::BN);
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, sm_count());
    return launch_pdl(kern, grid, C::THREADS, C::SMEM_BYTES, s, tA, tA32, tB, tC, p);
}

// The forms below (the last two 128 x 256, results stored by tensor stores or
// directly).
enum Form { kSmallTile = 0, kLargeTileByTensor = 1, kLargeTile = 2 };

}  // namespace

// Two tile shapes.  128 x 256: the least operand traffic per product, for
// everything that has rows.  64 x 128: twice the CTAs per group, for few rows,
// where the time is the stream of the weights and the SMs that take part in it;
// its stages hold two K blocks, so that the waits of the issuing and summing
// warps, which bound so small a block, are paid once for both (2 to 15 % of the
// times below).  The choice compares, per K block and in ns, the full waves of
// tiles, each at the rate of memory or of one CTA's loop, and the last partial one
// at the latter.  430 is the large tile's loop on streams that leave SMs idle
// (380 to 440 by the slope of K 4096, 8192 and 16384), 330 the small one's with one
// block per stage; with two it takes 200 to 270, so that the rule leans to the
// large tile where the two are close.  Measured with K 4096, N 1536 (small against
// large tiles): 8 rows over 8 experts 13.6 / 17.9 us, 16 over 16 24.2 / 22.0, 32 over
// 29 35.4 / 41.6, 4096 over 128 131 / 139, 8192 over 128 146 / 144, 512 over 8 14.0 /
// 19.2; the rule takes the smaller of each two.
cudaError_t launch_gemm_fp8_block(const GemmBlockArgs &a, cudaStream_t s) {
    const int64_t T = a.groups.total_rows, g = std::min<int64_t>(a.groups.num_groups, T);
    const int64_t sms = sm_count();
    auto cost = [&](int64_t bm, int64_t bn, int64_t loop_ns) {
        // m-blocks of g groups of about equal size: half of one is empty each
        const int64_t tiles = std::max(g, T / bm + g / 2) * ((a.N + bn - 1) / bn);
        const int64_t stream_ns = sms * bn * 128 / 6800;  // a wave's weights at 6.8 TB/s
        return tiles / sms * std::max(loop_ns, stream_ns) + (tiles % sms ? loop_ns : 0);
    };
    int tile = kSmallTile;
    // short reductions: a tile's results leave while the next one is summed, for
    // one stage of the ring (K 224: 90 us against 116 on 48816 x 3832; K 1536
    // 772 / 808 on 131072 x 4096; K 2480 97.2 / 97.8; K 4096 342 / 334; K 7168
    // 1554 / 1440, single launches)
    if (cost(64, 128, 330) >= cost(128, 256, 430))
        tile = a.K <= 20 * 128 ? kLargeTileByTensor : kLargeTile;
#ifdef MOEQ_FP8_BLOCK_TILE
    tile = MOEQ_FP8_BLOCK_TILE;  // test builds: one form for every size
#endif
    if (tile == kSmallTile) return run_block_gemm<BlockCfg<64, 128, 4, 8, false, 2>>(a, s);
    if (tile == kLargeTileByTensor) return run_block_gemm<BlockCfg<128, 256, 3, 8, true, 1>>(a, s);
    return run_block_gemm<BlockCfg<128, 256, 4, 8, false, 1>>(a, s);
}

}  // namespace moeq
