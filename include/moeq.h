/*
 * moeq: grouped mixture-of-experts low-precision kernels for one GB300 GPU
 * (sm_103a).  C ABI.
 *
 * Conventions shared by every call below
 * --------------------------------------
 * - Every pointer is a DEVICE pointer the caller owns (allocated with
 *   cudaMalloc, PyTorch, ...).  The library never allocates, frees or
 *   synchronises inside a compute call; each call only enqueues kernels on
 *   `stream` (a cudaStream_t; NULL = the legacy default stream) and returns.
 *   Pointers must be 16-byte aligned unless stated otherwise.
 * - Ragged expert groups ("grouped_matmul_rowwise_dynamic_scaled_fp8", Args
 *   a_offsets / expert_ids): group g = 0..num_active_experts-1 owns rows
 *   [offsets[g], offsets[g+1]) and uses expert expert_ids[g] (any order,
 *   need not be sorted or unique).  offsets are uint32 [G+1], expert_ids are
 *   int32 [G].  Empty groups write nothing.  Rows outside every group are
 *   never written.
 * - Padded scale rows ("max.nn.moe.NvMxf4f8Strategy", grouped_quantize:
 *   per-expert padding of the scales; "grouped_quantize_dynamic_scaled_fp4_async_kernel",
 *   scales_offsets): the block scales of group g live in logical scale rows
 *   [scales_offsets[g], scales_offsets[g+1]); scales_offsets[g] must be a
 *   multiple of 128 and leave room for ceil(r_g / 128) * 128 rows.
 *   moeq_padded_scale_offsets() builds the tightest such offsets.
 * - Block-scale layout (the tensor core's tiled layout; the pages leave it
 *   open): logical scales [rows, Kv] (Kv = K / block) are stored as 512-byte
 *   atoms of 128 rows x 4 columns; byte (r, c) of an atom is at
 *   (r % 32) * 16 + (r / 32) * 4 + c; atom (rb, kb) starts at
 *   (rb * ceil(Kv / 4) + kb) * 512.  Weight scales are one such buffer per
 *   expert, each ceil(N / 128) * ceil(Kv / 4) * 512 bytes.
 * - FP4 elements are packed two per byte, the lower-k element in the low
 *   nibble.
 * - Routed tokens ("Struct_ep_dispatch_mxfp4", execute, on one rank):
 *   moeq_route_topk turns per-token top-k expert ids into the group layout
 *   above (group e = expert e, every expert, stable order);
 *   moeq_grouped_amax_scale_topk and moeq_quantize_topk then read each token
 *   once and give the bytes of the row-level calls on the routed rows.
 * - Host threads.  Calls may be made concurrently from several host threads,
 *   on the same or different streams.  The only host state the library
 *   keeps is per-device launch set-up (SM count, kernel attributes applied,
 *   occupancy answers), computed once per device under an internal lock.
 *   moeq_last_cuda_error() is per host thread.  The device error word is
 *   shared by every call on a device.
 * - num_active_experts == 0 (or zero total rows) is MOEQ_OK and launches
 *   nothing.  max_tokens_per_expert is a sizing hint (the largest token
 *   count of any active expert): it picks launch shapes only, and groups larger than
 *   it are still computed in full.
 * - Errors.  Bad host arguments return MOEQ_ERR_INVALID_ARG before anything
 *   is launched (this includes a missing NVFP4 scale tensor, the pages'
 *   ValueError of prepare_swiglu_operands).  A shape or format that is not
 *   built returns MOEQ_ERR_UNSUPPORTED.  A launch failure returns
 *   MOEQ_ERR_CUDA (see moeq_last_cuda_error()).  Bad device-side data
 *   (non-monotone offsets, an expert id outside [0, num_experts), offsets
 *   past the buffers, a wait that timed out) never faults the GPU: the
 *   affected group is skipped and a sticky bit is set in the device error
 *   word, read with moeq_get_device_error().
 */
#ifndef MOEQ_H
#define MOEQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *moeq_stream_t; /* == cudaStream_t */

typedef enum {
    MOEQ_OK = 0,
    MOEQ_ERR_INVALID_ARG = 1,
    MOEQ_ERR_UNSUPPORTED = 2,
    MOEQ_ERR_CUDA = 3,
    MOEQ_ERR_DEVICE = 4
} moeq_status;

/* Quantized formats ("max.nn.moe.NvMxf4f8Strategy", is_nvfp4; the kernel of
 * "grouped_quantize_dynamic_scaled_fp4_async_kernel" quantizes to
 * NVFP4 / MXFP4 / MXFP8).
 *   NVFP4: E2M1 elements, 16-element blocks, E4M3 block scale, fp32
 *          per-expert tensor scale.
 *   MXFP4: E2M1 elements, 32-element blocks, E8M0 block scale.
 *   MXFP8: E4M3 elements, 32-element blocks, E8M0 block scale. */
typedef enum { MOEQ_NVFP4 = 0, MOEQ_MXFP4 = 1, MOEQ_MXFP8 = 2 } moeq_format;

/* Element types of the router's logits and of tokens and rows. */
typedef enum { MOEQ_BF16 = 0, MOEQ_FP16 = 1, MOEQ_FP32 = 2 } moeq_dtype;

/* Device error word bits (sticky until moeq_clear_device_error). */
#define MOEQ_DEVERR_BAD_OFFSETS 0x1u /* non-monotone or out-of-range offsets */
#define MOEQ_DEVERR_BAD_EXPERT 0x2u  /* expert id outside [0, num_experts)   */
#define MOEQ_DEVERR_SCALE_ROWS 0x4u  /* scale offsets unaligned / too small  */
#define MOEQ_DEVERR_TIMEOUT 0x8u     /* a pipeline wait gave up (~1 s)       */
#define MOEQ_DEVERR_BAD_INDEX 0x10u  /* gather index outside the input rows  */
#define MOEQ_DEVERR_BOUNDS 0x20u     /* debug builds: a store outside its buffer was skipped */

/* Per-expert NVFP4 tensor scale of the activations
 * ("grouped_quantize_dynamic_scaled_fp4_async_kernel": sf_tensor, the
 * per-expert tensor-wise scale factor, is a read-only input; this call
 * produces it).  tensor_scale_out[e] = fp32(amax_e / 2688), 2688 = 6 * 448,
 * amax_e = max |in| over all rows of all groups routed to expert e; experts
 * with no rows or an all-zero input get 1.0.
 *   in            bf16 [total_rows, K], row stride in_row_stride elements.
 *   row_offsets   uint32 [G+1]; expert_ids int32 [G].
 *   tensor_scale_out  fp32 [num_experts], fully overwritten.
 * K must be a multiple of 8; in_row_stride a multiple of 8, >= K. */
moeq_status moeq_grouped_amax_scale(const void *in, int64_t in_row_stride,
                                    int64_t total_rows, int64_t K,
                                    const uint32_t *row_offsets,
                                    const int32_t *expert_ids,
                                    float *tensor_scale_out,
                                    int32_t num_experts,
                                    int32_t num_active_experts,
                                    moeq_stream_t stream);

/* Grouped activation quantizer ("grouped_quantize_dynamic_scaled_fp4_async_kernel":
 * each block of work finds its expert by binary search on row_offsets /
 * scales_offsets and quantizes that expert's BF16 rows; "max.nn.moe.NvMxf4f8Strategy",
 * grouped_quantize).
 *   in            bf16 [total_rows, K], row stride in_row_stride elements.
 *   out           NVFP4 / MXFP4: [total_rows, K/2] packed; MXFP8: [total_rows, K].
 *   scales        tiled block-scale buffer of scale_rows_total logical rows
 *                 x K/16 (NVFP4) or K/32 (MX) columns.  For group g the rows
 *                 [scales_offsets[g], scales_offsets[g] + r_g) get the scales of
 *                 its rows and the rows up to scales_offsets[g] + ceil(r_g/128)*128
 *                 are zeroed; any further rows and rows >= scales_offsets[G]
 *                 are untouched.
 *   tensor_scale  fp32 [num_experts] raw (dequantization-direction) scale s_e
 *                 (NVFP4 only, required; ignored for MX).
 * Per block (NVFP4): inv = 1/s_e; sb = E4M3((amax * inv) / 6);
 * q = E2M1(x * (inv / sb)), all zero when sb == 0.  MX: scale code
 * c = clamp(floor(log2 amax) - emax + 127, 0, 254) (emax 8 for E4M3, 2 for
 * E2M1); q = elem(x * 2^(127-c)); an all-zero block is all +0 with c = 0.
 * All rounding is to nearest even, saturating.  K must be a multiple of 128;
 * scale_rows_total a multiple of 128. */
moeq_status moeq_grouped_quantize(moeq_format fmt, const void *in,
                                  int64_t in_row_stride, int64_t total_rows,
                                  int64_t K, uint8_t *out, uint8_t *scales,
                                  int64_t scale_rows_total,
                                  const uint32_t *row_offsets,
                                  const uint32_t *scales_offsets,
                                  const int32_t *expert_ids,
                                  const float *tensor_scale,
                                  int32_t num_experts,
                                  int32_t max_tokens_per_expert,
                                  int32_t num_active_experts,
                                  moeq_stream_t stream);

/* Gather-fused variants ("max.nn.moe.NvMxf4f8Strategy", grouped_quantize:
 * the indices and indices_divisor arguments).  Reading adopted: the rows
 * being quantized are gathered from the input, quantized row t reading input
 * row indices[t] / indices_divisor (e.g. indices = the expert-sorted
 * positions token * top_k + slot and indices_divisor = top_k, so the MoE
 * permutation needs no separate copy).  Everything else is exactly
 * moeq_grouped_amax_scale / moeq_grouped_quantize on the gathered rows.
 *   in          bf16 [in_rows, K], row stride in_row_stride elements.
 *   indices     int32 [total_rows] (device); indices_divisor >= 1.
 *   total_rows  number of quantized rows (row_offsets index these).
 * An index whose input row falls outside [0, in_rows) skips that row and
 * sets MOEQ_DEVERR_BAD_INDEX. */
moeq_status moeq_grouped_amax_scale_gather(const void *in, int64_t in_row_stride,
                                           int64_t in_rows, int64_t K,
                                           const int32_t *indices, int32_t indices_divisor,
                                           int64_t total_rows, const uint32_t *row_offsets,
                                           const int32_t *expert_ids, float *tensor_scale_out,
                                           int32_t num_experts, int32_t num_active_experts,
                                           moeq_stream_t stream);

moeq_status moeq_grouped_quantize_gather(moeq_format fmt, const void *in, int64_t in_row_stride,
                                         int64_t in_rows, int64_t K, const int32_t *indices,
                                         int32_t indices_divisor, int64_t total_rows,
                                         uint8_t *out, uint8_t *scales, int64_t scale_rows_total,
                                         const uint32_t *row_offsets,
                                         const uint32_t *scales_offsets,
                                         const int32_t *expert_ids, const float *tensor_scale,
                                         int32_t num_experts, int32_t max_tokens_per_expert,
                                         int32_t num_active_experts, moeq_stream_t stream);

/* scales_offsets[g] = sum_{h<g} ceil((row_offsets[h+1]-row_offsets[h]) / 128) * 128,
 * g = 0..G (uint32 [G+1], device).  The tightest padding accepted by the
 * calls above. */
moeq_status moeq_padded_scale_offsets(const uint32_t *row_offsets,
                                      uint32_t *scales_offsets,
                                      int32_t num_active_experts,
                                      moeq_stream_t stream);

/* Grouped rowwise-scaled FP8 matmul ("grouped_matmul_rowwise_dynamic_scaled_fp8",
 * description and Args):
 *   c[t, n] = bf16( (sum_k a[t,k] * b[expert_ids[g], n, k]) * a_scales[t]
 *                   * b_scales[expert_ids[g], n] )
 * accumulated in fp32 by the tensor cores, the two scales applied once after
 * the reduction (acc * a_scale first, then * b_scale), round to nearest even.
 *   c         bf16 [total_tokens, N]
 *   a         E4M3 [total_tokens, K]
 *   b         E4M3 [num_experts, N, K] (K innermost: the page accepts only transposed b)
 *   a_scales  fp32 [total_tokens];  b_scales fp32 [num_experts, N]
 * K % 128 == 0, N % 16 == 0. */
moeq_status moeq_grouped_matmul_rowwise_fp8(
    void *c, const uint8_t *a, const uint8_t *b, const float *a_scales,
    const float *b_scales, const uint32_t *a_offsets,
    const int32_t *expert_ids, int64_t total_tokens, int64_t N, int64_t K,
    int32_t num_experts, int32_t max_tokens_per_expert,
    int32_t num_active_experts, moeq_stream_t stream);

/* Grouped block-scaled matmul with per-expert epilogue scales
 * ("max.nn.moe.NvMxf4f8Strategy", grouped_matmul: a grouped block-scaled
 * matmul with one scale per expert, applied in the matmul epilogue):
 *   c[t, n] = bf16( expert_scales[e] * sum_k (qa[t,k] * sa[t,k/v]) * (qb[e,n,k] * sb[e,n,k/v]) )
 * with e = expert_ids[g], v = 16 (NVFP4) or 32 (MXFP8, MXFP4).
 *   a      NVFP4 / MXFP4: packed [total_tokens, K/2]; MXFP8: [total_tokens, K]
 *   a_sf   tiled scales, scale_rows_total rows; row t of group g uses
 *          scale row a_scales_offsets[g] + (t - a_offsets[g])
 *   b      NVFP4 / MXFP4: packed [num_experts, N, K/2]; MXFP8: [num_experts, N, K]
 *   b_sf   per-expert tiled scales (see the layout above)
 *   expert_scales  fp32 [num_experts]; required for NVFP4, NULL means 1 for MX.
 * NVFP4 and MXFP4: K % 256 == 0; MXFP8: K % 128 == 0; N % 128 == 0. */
moeq_status moeq_grouped_matmul_blockscaled(
    moeq_format fmt, void *c, const uint8_t *a, const uint8_t *a_sf,
    const uint8_t *b, const uint8_t *b_sf, const float *expert_scales,
    const uint32_t *a_offsets, const uint32_t *a_scales_offsets,
    const int32_t *expert_ids, int64_t total_tokens, int64_t scale_rows_total,
    int64_t N, int64_t K, int32_t num_experts, int32_t max_tokens_per_expert,
    int32_t num_active_experts, moeq_stream_t stream);

/* Chained SwiGLU + NVFP4 requantization ("max.nn.moe.NvMxf4f8Strategy",
 * fused_silu_quantize: the gated activation, then quantization; the
 * SiLU-output scale is passed raw and inverted inside, as
 * prepare_swiglu_operands requires).
 *   y      bf16 [total_tokens, 2I]: column 2j = gate_j, 2j+1 = up_j
 *   h_j    = silu(gate_j) * up_j in fp32, silu(g) = g * sigma(g) with the
 *            library's own deterministic sigma, each step one IEEE fp32
 *            operation or one fused multiply-add:
 *              e = exp(-|g|): Cody-Waite reduction (ln 2 split into a
 *                  16-bit head and an fp32 tail, n from one FMA with the
 *                  1.5 * 2^23 shift), degree-7 Taylor polynomial by Horner
 *                  in FMAs, times 2^n (2^n taken as 0 for n < -126);
 *              d = 1 + e;  r = 1 / d by three Newton steps in FMAs
 *                  (q = 1 - d r, r = r + r q) from 24/17 - 8/17 d;
 *              sigma = r for g >= 0, e * r otherwise.
 *            CUDA's expf and IEEE division are not used.
 *   c_packed  NVFP4 [total_tokens, I/2];  c_sf tiled scales [scale_rows_total
 *            rows x I/16], padded per expert exactly like moeq_grouped_quantize
 *   out_tensor_scale  fp32 [num_experts] raw s_e (required).
 * I % 64 == 0. */
moeq_status moeq_swiglu_quantize(uint8_t *c_packed, uint8_t *c_sf,
                                 const void *y, const float *out_tensor_scale,
                                 const uint32_t *a_offsets,
                                 const uint32_t *a_scales_offsets,
                                 const int32_t *expert_ids,
                                 int64_t total_tokens,
                                 int64_t scale_rows_total, int64_t I,
                                 int32_t num_experts,
                                 int32_t max_tokens_per_expert,
                                 int32_t num_active_experts,
                                 moeq_stream_t stream);

/* Chained SwiGLU + MX requantization ("max.nn.moe.NvMxf4f8Strategy": the
 * strategy handles NVFP4, MXFP4 or MXFP8; fused_silu_quantize applies the
 * gated activation and then quantizes, read here as quantizing in the
 * strategy's format; MX formats carry no tensor scale).
 *   h as in moeq_swiglu_quantize, then per 32-element block of h the MX rule
 *   of moeq_grouped_quantize: c = clamp(floor(log2 amax) - emax + 127, 0, 254)
 *   (amax of the fp32 h values), q = elem(h * 2^(127-c)), an all-zero block
 *   all +0 with c = 0.
 *   fmt     MOEQ_MXFP4 (E2M1, c_q [total_tokens, I/2] packed) or MOEQ_MXFP8
 *           (E4M3, c_q [total_tokens, I]).
 *   c_sf    tiled E8M0 scales [scale_rows_total rows x I/32], padded per
 *           expert like moeq_grouped_quantize.
 * I % 128 == 0. */
moeq_status moeq_swiglu_quantize_mx(moeq_format fmt, uint8_t *c_q, uint8_t *c_sf,
                                    const void *y, const uint32_t *a_offsets,
                                    const uint32_t *a_scales_offsets,
                                    const int32_t *expert_ids, int64_t total_tokens,
                                    int64_t scale_rows_total, int64_t I,
                                    int32_t num_experts, int32_t max_tokens_per_expert,
                                    int32_t num_active_experts, moeq_stream_t stream);

/* Fused grouped NVFP4 matmul + SwiGLU + NVFP4 requantization in one kernel
 * ("max.nn.moe.NvMxf4f8Strategy", grouped_matmul_swiglu: equivalent to
 * grouped_matmul followed by fused_silu_quantize; its (c_packed,
 * c_swiglu_scales) match the chained path byte for byte with a bf16
 * rounding where the chained path has a bf16 tensor).
 * Computes, with no bf16 tensor in memory, exactly
 *   moeq_grouped_matmul_blockscaled(NVFP4, y, ...) ; moeq_swiglu_quantize(..., y, ...)
 * and writes the same bytes.  b is [num_experts, 2I, K/2] with gate/up rows
 * interleaved (row 2j = gate_j, row 2j+1 = up_j); b_sf its per-expert tiled
 * scales.  expert_scales and out_tensor_scale are required.
 *   a_row_scales  optional bf16 [total_tokens] (NULL = none; grouped_matmul_swiglu:
 *            one bf16 scale per row, applied with the expert scale ahead
 *            of the SwiGLU): gate and up become
 *            bf16((acc * expert_scale) * a_row_scale[t]), two fp32 multiplies
 *            in that order.  With row scales there is no chained counterpart.
 * K % 256 == 0, I % 64 == 0. */
moeq_status moeq_grouped_matmul_swiglu(
    uint8_t *c_packed, uint8_t *c_sf, const uint8_t *a, const uint8_t *a_sf,
    const uint8_t *b, const uint8_t *b_sf, const float *expert_scales,
    const float *out_tensor_scale, const void *a_row_scales, const uint32_t *a_offsets,
    const uint32_t *a_scales_offsets, const int32_t *expert_ids,
    int64_t total_tokens, int64_t scale_rows_total, int64_t I, int64_t K,
    int32_t num_experts, int32_t max_tokens_per_expert,
    int32_t num_active_experts, moeq_stream_t stream);

/* Fused grouped MX matmul + SwiGLU + MX requantization in one kernel: the
 * MX counterpart of moeq_grouped_matmul_swiglu (same reading of the
 * strategy: MXFP4 or MXFP8 throughout).  Computes, with no bf16 tensor in
 * memory, exactly
 *   moeq_grouped_matmul_blockscaled(fmt, y, ...) ; moeq_swiglu_quantize_mx(fmt, ..., y, ...)
 * and writes the same bytes.  a / a_sf / b / b_sf as for
 * moeq_grouped_matmul_blockscaled(fmt) with N = 2I (gate/up rows of b
 * interleaved); expert_scales optional (NULL = 1).
 * MXFP4: K % 256 == 0; MXFP8: K % 128 == 0; I % 128 == 0. */
moeq_status moeq_grouped_matmul_swiglu_mx(
    moeq_format fmt, uint8_t *c_q, uint8_t *c_sf, const uint8_t *a, const uint8_t *a_sf,
    const uint8_t *b, const uint8_t *b_sf, const float *expert_scales,
    const uint32_t *a_offsets, const uint32_t *a_scales_offsets, const int32_t *expert_ids,
    int64_t total_tokens, int64_t scale_rows_total, int64_t I, int64_t K,
    int32_t num_experts, int32_t max_tokens_per_expert, int32_t num_active_experts,
    moeq_stream_t stream);

/* ---- weight preparation ("max.nn.moe.NvMxf4f8Strategy", prepare_weight_scales:
 * block scales rearranged into the kernel's layout).  Run once per weight,
 * off the per-step path.  Every pointer is a caller-owned device pointer;
 * the calls only enqueue work on `stream`.  batch, rows, kv / row_bytes == 0
 * is MOEQ_OK and a no-op; negative sizes or NULL pointers (with a non-empty
 * call) return MOEQ_ERR_INVALID_ARG before any launch. */

/* Logical -> tiled block-scale layout, for `batch` independent matrices
 * (e.g. one per expert).
 *   logical  uint8 [batch, rows, kv], row-major, kv = K / block size
 *   tiled    uint8 [batch, ceil(rows / 128) * ceil(kv / 4) * 512]: matrix b starts at byte
 *            b * ceil(rows / 128) * ceil(kv / 4) * 512; inside it scale (r, c)
 *            sits in the 512-byte atom (r / 128, c / 4) (atoms row-block-major)
 *            at byte (r % 32) * 16 + ((r / 32) % 4) * 4 + c % 4 -- the layout
 *            every block-scaled call reads and writes.
 * Bytes of the tiled buffer that hold no logical scale are written 0. */
moeq_status moeq_sf_swizzle(uint8_t *tiled, const uint8_t *logical, int64_t batch,
                            int64_t rows, int64_t kv, moeq_stream_t stream);

/* Tiled -> logical (the inverse of moeq_sf_swizzle; padding is not read
 * into the output, which holds exactly batch * rows * kv bytes). */
moeq_status moeq_sf_unswizzle(uint8_t *logical, const uint8_t *tiled, int64_t batch,
                              int64_t rows, int64_t kv, moeq_stream_t stream);

/* Gate/up interleave of the fused SwiGLU GEMM's weight: out[b, 2j, :] =
 * gate[b, j, :] and out[b, 2j + 1, :] = up[b, j, :] for rows of row_bytes
 * bytes (packed weight rows, K / 2 bytes for E2M1; or logical scale rows,
 * kv bytes, then moeq_sf_swizzle with 2 * rows rows).
 *   gate, up uint8 [batch, rows, row_bytes];  out uint8 [batch, 2 * rows, row_bytes]
 * out must not overlap the inputs. */
moeq_status moeq_interleave_gate_up(uint8_t *out, const uint8_t *gate, const uint8_t *up,
                                    int64_t batch, int64_t rows, int64_t row_bytes,
                                    moeq_stream_t stream);

/* Expert dispatch on one rank ("Struct_ep_dispatch_mxfp4", execute: the
 * row_offsets, expert_ids and src_info outputs and the MXFP4 tokens; with a
 * single rank the all-to-all exchange is the identity and is not built).
 *
 * moeq_route_topk routes every choice i = t * top_k + k of topk_ids to the
 * group of its expert.  Group e is expert e for all e in [0, num_experts),
 * empty groups included; a group's rows hold its choices in increasing i
 * (a stable order: the page's atomic counters leave the order open).
 *   topk_ids        int32 [num_tokens, top_k] (device), expert of each choice.
 *   row_offsets     u32 [num_experts + 1] (out)
 *   expert_ids      int32 [num_experts] (out): 0 .. num_experts - 1
 *   src_info        int32 [num_tokens * top_k] (out): row r holds choice
 *                   src_info[r] (token src_info[r] / top_k); entries past
 *                   row_offsets[num_experts] are not written.
 *   dst_info        int32 [num_tokens * top_k] (out, may be NULL): the row of
 *                   choice i (the inverse of src_info), -1 for a dropped
 *                   choice.
 *   scales_offsets  u32 [num_experts + 1] (out, may be NULL): with
 *                   slot_rows == 0 the padded prefix of ceil(r_e / 128) * 128
 *                   (as moeq_padded_scale_offsets); with slot_rows > 0 (a
 *                   multiple of 128) the fixed-stride slots e * slot_rows of
 *                   the page's scale-slot fusion (fuse_a_scale_preshuffle,
 *                   slot stride max_padded_M).
 * A choice whose expert id lies outside [0, num_experts) is dropped and sets
 * MOEQ_DEVERR_BAD_EXPERT.  Limits: 1 <= num_experts <= 1024 (else
 * MOEQ_ERR_UNSUPPORTED), num_tokens * top_k < 2^31.  One CTA on one SM; no
 * memory besides the outputs. */
moeq_status moeq_route_topk(const int32_t *topk_ids, int64_t num_tokens, int32_t top_k,
                            int32_t num_experts, uint32_t *row_offsets, int32_t *expert_ids,
                            int32_t *src_info, int32_t *dst_info, uint32_t *scales_offsets,
                            int32_t slot_rows, moeq_stream_t stream);

/* Token-major quantization of routed tokens: the bytes of
 * moeq_grouped_quantize_gather(fmt, tokens, indices = src_info,
 * indices_divisor = top_k, groups = all num_experts experts, row_offsets,
 * scales_offsets, expert_ids = 0..E-1, tensor_scale) -- the same NVFP4 /
 * MXFP4 / MXFP8 rule per routed row, padding scale rows zero -- but each
 * token row is read once and written to its routed rows dst_info[t * top_k
 * + j] (MX formats quantize it once; NVFP4 shares the loads and block amax
 * across the choices' tensor scales).
 *   tokens       bf16 [num_tokens, K], row stride token_stride; K % 128 == 0.
 *   topk_ids, dst_info  int32 [num_tokens * top_k] (from moeq_route_topk).
 *   row_offsets, scales_offsets  u32 [num_experts + 1] (from moeq_route_topk).
 *   tensor_scale fp32 [num_experts] raw per-expert scales (NVFP4 only).
 *   out          [num_tokens * top_k, K / 2] (FP4) or [.., K] (MXFP8).
 *   scales       tiled block scales of scale_rows_total logical rows.
 * top_k <= 8 (else MOEQ_ERR_UNSUPPORTED).  A group whose scale rows do not
 * fit is skipped and sets MOEQ_DEVERR_SCALE_ROWS. */
moeq_status moeq_quantize_topk(moeq_format fmt, const void *tokens, int64_t token_stride,
                               int64_t num_tokens, int64_t K, const int32_t *topk_ids,
                               int32_t top_k, const int32_t *dst_info,
                               const uint32_t *row_offsets, const uint32_t *scales_offsets,
                               const float *tensor_scale, int32_t num_experts, uint8_t *out,
                               uint8_t *scales, int64_t scale_rows_total, moeq_stream_t stream);

/* Per-expert NVFP4 tensor scales from tokens and their top-k expert ids:
 * tensor_scale_out[e] = amax_e / (6 * 448) (1 when amax_e == 0), amax_e the
 * max |x| over the tokens with a choice of expert e -- the value
 * moeq_grouped_amax_scale gives over the routed rows
 * ("grouped_quantize_dynamic_scaled_fp4_async_kernel": the per-expert tensor
 * scale), but each token row is read once instead of once per choice.
 *   tokens      bf16 [num_tokens, K], row stride token_stride elements.
 *   topk_ids    int32 [num_tokens, top_k] (device).
 *   tensor_scale_out  fp32 [num_experts] (out).
 * An id outside [0, num_experts) is skipped and sets MOEQ_DEVERR_BAD_EXPERT. */
moeq_status moeq_grouped_amax_scale_topk(const void *tokens, int64_t token_stride,
                                         int64_t num_tokens, int64_t K, const int32_t *topk_ids,
                                         int32_t top_k, float *tensor_scale_out,
                                         int32_t num_experts, moeq_stream_t stream);

/* Scale rows that moeq_dispatch_mxfp4 needs: num_experts * slot_rows with
 * slot_rows > 0, else the largest possible padded total,
 * floor((num_tokens * top_k + 127 * num_experts) / 128) * 128.  Host only. */
int64_t moeq_dispatch_scale_rows(int64_t num_tokens, int32_t top_k, int32_t num_experts,
                                 int32_t slot_rows);

/* moeq_route_topk, then MXFP4 quantization of the routed rows (routed row r
 * is token src_info[r] / top_k), token-major (moeq_quantize_topk: each
 * token quantized once and stored to its top_k rows), in stream order.
 *   tokens          bf16 [num_tokens, hidden], row stride token_stride
 *                   elements; hidden a multiple of 128.
 *   out             uint8 [num_tokens * top_k, hidden / 2] packed E2M1
 *                   (rows past the routed count are not written).
 *   scales          tiled E8M0 block scales of scale_rows_total logical rows
 *                   of hidden / 32 scales; scale_rows_total >=
 *                   moeq_dispatch_scale_rows(...) and a multiple of 128.
 *   row_offsets, expert_ids, src_info, dst_info, scales_offsets: as
 *                   moeq_route_topk (dst_info and scales_offsets required
 *                   here).  top_k <= 8.
 * With slot_rows > 0 a group larger than slot_rows is not quantized and
 * sets MOEQ_DEVERR_SCALE_ROWS. */
moeq_status moeq_dispatch_mxfp4(const void *tokens, int64_t token_stride, int64_t num_tokens,
                                int64_t hidden, const int32_t *topk_ids, int32_t top_k,
                                int32_t num_experts, uint8_t *out, uint8_t *scales,
                                int64_t scale_rows_total, uint32_t *row_offsets,
                                int32_t *expert_ids, int32_t *src_info, int32_t *dst_info,
                                uint32_t *scales_offsets, int32_t slot_rows,
                                moeq_stream_t stream);

/* ---- the router, tokens to rows and back (with gradients), FP8 with 128-blocks
 *
 * moeq_gate_topk: the top_k largest logits of each token, largest first, ties
 * to the lowest index, and their softmax weights.  With x a token's logits,
 * m = max x, i_r its choices:
 *   normalize == 0:  w_r = scale * exp(x_{i_r} - m) / sum over all experts of exp(x - m)
 *   normalize != 0:  w_r = scale * exp(x_{i_r} - m) / sum over the choices of exp(x - m)
 * fp32 throughout: d = x - m is rounded (|d| 2^-24 of the result), exp(d) of the rounded
 * d within 2 + 1.2 |d| ulp.
 *   logits      dtype [num_tokens, num_experts], row stride logit_stride elements.
 *   topk_ids    int32 [num_tokens, top_k] (out);  weights fp32 [num_tokens, top_k] (out).
 * A logit of -inf (a masked expert) or NaN is never chosen; a token with fewer
 * than top_k others gets id -1 and weight 0 in the places left over, which
 * moeq_route_topk drops (setting MOEQ_DEVERR_BAD_EXPERT).  A NaN or +inf logit
 * makes all weights of a token that has a choice NaN, in the places left over too;
 * a token without a choice has weights 0.
 * 1 <= top_k <= num_experts; num_experts <= 1024 and top_k <= 32 (else
 * MOEQ_ERR_UNSUPPORTED). */
moeq_status moeq_gate_topk(moeq_dtype dtype, const void *logits, int64_t logit_stride,
                           int64_t num_tokens, int32_t num_experts, int32_t top_k,
                           int32_t normalize, float scale, int32_t *topk_ids, float *weights,
                           moeq_stream_t stream);

/* Gradient of moeq_gate_topk's weights (the choice is taken as fixed): with p
 * the softmax over all experts, q = w / scale and g_j = sum over r with
 * i_r = j of scale * d_weights_r,
 *   normalize == 0:  d_logits = p * (g - <p, g>)
 *   normalize != 0:  d_logits_{i_r} = scale * q_r * (d_weights_r - <q, d_weights>), 0 elsewhere.
 * A token without a choice gets 0; a NaN or +inf logit makes a token's gradient NaN
 * (with normalize that of the chosen).
 *   logits, topk_ids  as given to and returned by moeq_gate_topk: a token's ids are
 *               distinct (an id of -1 is skipped; any other id outside the experts too,
 *               and sets MOEQ_DEVERR_BAD_EXPERT).
 *   d_weights   fp32 [num_tokens, top_k];  d_logits dtype [num_tokens, num_experts] (out). */
moeq_status moeq_gate_topk_grad(moeq_dtype dtype, const void *logits, int64_t logit_stride,
                                int64_t num_tokens, int32_t num_experts, int32_t top_k,
                                int32_t normalize, float scale, const int32_t *topk_ids,
                                const float *d_weights, void *d_logits, moeq_stream_t stream);

/* The router with scores, a balance bias and groups of experts.  With x a token's
 * logits, s_j = sigmoid(x_j) or the softmax of x, c_j = s_j + bias_j:
 *   the experts are num_groups groups of consecutive ones; a group's value is its
 *   largest c (MOEQ_GROUP_MAX), or the sum of its two largest (MOEQ_GROUP_TOP2; of one
 *   usable expert alone, that one's); of the topk_groups groups of the largest values
 *   (ties: the lowest index) the top_k experts of the largest c (ties: the lowest
 *   index) are chosen, the largest first;
 *   normalize == 0:  w_r = scale * s_{i_r}
 *   normalize != 0:  w_r = scale * s_{i_r} / sum over the choices of s  (0 where it is 0)
 * The bias decides the choice and does not enter the weights; without one (NULL) c is
 * ordered as the logits are.  The order is that of the real values, whatever their rounding
 * to fp32, of experts' c and of groups' sums alike, where they are further apart than 2^-42 of
 * the largest score or bias that is in them; what is closer may fall either way, and
 * equal logits with equal biases tie (a score below 2^-126 counts as 0).  Weights are
 * fp32, from s within 4 ulp (sigmoid; a score below 2^-126 has the few bits that fp32 has
 * there) or as in moeq_gate_topk.
 *   logits      dtype [num_tokens, num_experts], row stride logit_stride elements.
 *   bias        fp32 [num_experts] or NULL.
 *   topk_ids    int32 [num_tokens, top_k] (out);  weights fp32 [num_tokens, top_k] (out).
 * A logit of -inf or NaN, and with a bias one whose c is (a bias of -inf or NaN), is never
 * chosen; places left over get id -1 and weight 0.  A NaN logit makes all weights of a
 * token that has a choice NaN; for a softmax a +inf logit does too, and such a token's
 * choice goes by its logits, without the bias.
 * num_groups divides num_experts; 1 <= topk_groups <= num_groups; 1 <= top_k <=
 * topk_groups * (num_experts / num_groups).  num_experts <= 1024, top_k <= 32,
 * num_groups <= 32 and, with P the power of two from num_groups on, at most 32
 * experts for each of the 32 / P lanes that a group has, num_experts / num_groups <=
 * 1024 / P (else MOEQ_ERR_UNSUPPORTED). */
typedef enum { MOEQ_SCORE_SOFTMAX = 0, MOEQ_SCORE_SIGMOID = 1 } moeq_score;
typedef enum { MOEQ_GROUP_MAX = 0, MOEQ_GROUP_TOP2 = 1 } moeq_group_score;
moeq_status moeq_gate_group_topk(moeq_dtype dtype, const void *logits, int64_t logit_stride,
                                 int64_t num_tokens, int32_t num_experts, const float *bias,
                                 moeq_score score, int32_t num_groups, int32_t topk_groups,
                                 moeq_group_score group_score, int32_t top_k, int32_t normalize,
                                 float scale, int32_t *topk_ids, float *weights,
                                 moeq_stream_t stream);

/* Gradient of moeq_gate_group_topk's weights (the choice is taken as fixed; the bias has
 * none): with q = w / scale and g_r = scale * d_weights_r,
 *   sigmoid, normalize == 0:  d_logits_{i_r} = g_r * s (1 - s)
 *   sigmoid, normalize != 0:  d_logits_{i_r} = q_r * (g_r - <q, g>) * (1 - s)
 *   softmax, normalize != 0:  d_logits_{i_r} = q_r * (g_r - <q, g>)
 * and 0 elsewhere: only the chosen logits are read, after a row was zeroed, so that
 * d_logits may not lie over logits.  Softmax without normalize is moeq_gate_topk_grad.
 * Arguments as there. */
moeq_status moeq_gate_group_topk_grad(moeq_dtype dtype, const void *logits, int64_t logit_stride,
                                      int64_t num_tokens, int32_t num_experts, moeq_score score,
                                      int32_t top_k, int32_t normalize, float scale,
                                      const int32_t *topk_ids, const float *d_weights,
                                      void *d_logits, moeq_stream_t stream);

/* Tokens sorted by expert: rows[dst_info[t, j]] = weights[t, j] * tokens[t].
 *   tokens    dtype [num_tokens, hidden], row stride token_stride elements.
 *   dst_info  int32 [num_tokens, top_k] (from moeq_route_topk): the row of each choice,
 *             -1 for a dropped one; any other value outside [0, total_rows) is skipped
 *             and sets MOEQ_DEVERR_BAD_INDEX.
 *   weights   fp32 [num_tokens, top_k], or NULL: the rows are copies.
 *   rows      dtype [total_rows, hidden] (out); rows that no choice has are not written.
 * Here and in the three calls below products and sums are fp32, rounded once when stored;
 * sums over the choices run in their order (no atomics).  hidden * sizeof(dtype) and
 * token_stride * sizeof(dtype) are multiples of 16; top_k <= 32, hidden < 2^24 (else
 * MOEQ_ERR_UNSUPPORTED). */
moeq_status moeq_permute_topk(moeq_dtype dtype, const void *tokens, int64_t token_stride,
                              int64_t num_tokens, int64_t hidden, const int32_t *dst_info,
                              int32_t top_k, const float *weights, void *rows, int64_t total_rows,
                              moeq_stream_t stream);

/* Gradient of moeq_permute_topk:
 *   d_tokens[t] = sum over j of weights[t, j] * d_rows[dst_info[t, j]]   (weights NULL: 1)
 *   d_weights[t, j] = <tokens[t], d_rows[dst_info[t, j]]>, 0 for a dropped choice.
 * d_weights (fp32 [num_tokens, top_k]) may be NULL; tokens is read for it only. */
moeq_status moeq_permute_topk_grad(moeq_dtype dtype, const void *d_rows, int64_t total_rows,
                                   int64_t num_tokens, int64_t hidden, const int32_t *dst_info,
                                   int32_t top_k, const float *weights, void *d_tokens,
                                   const void *tokens, int64_t token_stride, float *d_weights,
                                   moeq_stream_t stream);

/* Rows back to their tokens: out[t] = sum over j of weights[t, j] * rows[dst_info[t, j]]
 * (weights NULL: 1; dropped choices add nothing, a token with none is 0).
 *   rows dtype [total_rows, hidden];  out dtype [num_tokens, hidden]. */
moeq_status moeq_combine_topk(moeq_dtype dtype, const void *rows, int64_t total_rows,
                              int64_t num_tokens, int64_t hidden, const int32_t *dst_info,
                              int32_t top_k, const float *weights, void *out,
                              moeq_stream_t stream);

/* Gradient of moeq_combine_topk:
 *   d_rows[dst_info[t, j]] = weights[t, j] * d_out[t]   (weights NULL: 1)
 *   d_weights[t, j] = <d_out[t], rows[dst_info[t, j]]>, 0 for a dropped choice.
 * d_out has row stride d_out_stride elements; d_rows must not overlap rows; d_weights may be
 * NULL, rows is read for it only. */
moeq_status moeq_combine_topk_grad(moeq_dtype dtype, const void *d_out, int64_t d_out_stride,
                                   int64_t num_tokens, int64_t hidden, const int32_t *dst_info,
                                   int32_t top_k, const float *weights, void *d_rows,
                                   int64_t total_rows, const void *rows, float *d_weights,
                                   moeq_stream_t stream);

/* FP8 with one fp32 scale per block of 128 (the last block of a row may be
 * shorter).  Per block: s = max(amax / 448, 2^-126), q = E4M3(x * (1 / s)), each
 * step one fp32 operation, round to nearest even, saturating; q * s stands for x.
 * A NaN stays a NaN code of its element alone; an infinity gives its block an
 * infinite scale and itself a NaN code.  K % 16 == 0.
 *   in      bf16 [rows, K], row stride in_row_stride elements (a multiple of 8).
 *   out     E4M3 [rows, K];  scales fp32 [rows, ceil(K / 128)]. */
moeq_status moeq_quantize_fp8_block(const void *in, int64_t in_row_stride, int64_t rows, int64_t K,
                                    uint8_t *out, float *scales, moeq_stream_t stream);

/* The same of routed tokens: row dst_info[t, j] of out and scales is token t's
 * (each token read and quantized once).  dst_info, top_k and rows outside
 * [0, total_rows) as in moeq_permute_topk. */
moeq_status moeq_quantize_fp8_block_topk(const void *tokens, int64_t token_stride,
                                         int64_t num_tokens, int64_t K, const int32_t *dst_info,
                                         int32_t top_k, uint8_t *out, float *scales,
                                         int64_t total_rows, moeq_stream_t stream);

/* The same of h = silu(gate) * up (fp32, as in moeq_swiglu_quantize; not rounded
 * in between): y bf16 [rows, 2 I], column 2j = gate_j, 2j+1 = up_j; out E4M3
 * [rows, I]; scales fp32 [rows, ceil(I / 128)].  I % 16 == 0. */
moeq_status moeq_swiglu_quantize_fp8_block(const void *y, int64_t rows, int64_t I, uint8_t *out,
                                           float *scales, moeq_stream_t stream);

/* The same of weights, one scale per 128 x 128 block: w bf16 [num_experts, N, K];
 * out E4M3 of that shape; scales fp32 [num_experts, ceil(N / 128), ceil(K / 128)]. */
moeq_status moeq_quantize_fp8_block_weight(const void *w, int64_t num_experts, int64_t N, int64_t K,
                                           uint8_t *out, float *scales, moeq_stream_t stream);

/* ---- before a layer: the residual's addition, the root-mean-square norm and FP8
 *
 * For each row, of one dtype throughout:
 *   h = x + residual, rounded to the dtype (the new residual stream; without a
 *       residual h is x and is not written)
 *   rstd = 1 / sqrt(mean of h^2 + eps),  v = (h * rstd) * weight
 *   y = v, rounded to the dtype;  q, scales = v in E4M3 by the rule of
 *       moeq_quantize_fp8_block, from fp32 (not from y)
 * fp32 throughout, the squares' sum too (squares past its range give an infinite sum, those
 * below 2^-126 lose bits).
 *   x, residual dtype [rows, K], row strides x_stride, residual_stride elements.
 *   weight      dtype [K].
 *   h, y        dtype [rows, K] (out); h required with a residual and only then.
 *   q           E4M3 [rows, K] (out);  scales (out) fp32 [rows, ceil(K / 128)], or, with
 *               row_scales != 0, one for each row, fp32 [rows] (the operands of
 *               moeq_grouped_matmul_fp8_block and moeq_grouped_matmul_rowwise_fp8).
 *   rstd        fp32 [rows] (out), for the gradient.
 * y, q with scales, and rstd may be NULL, not all of them.  h and y, two buffers, may be
 * x's or the residual's own (the same rows at the same stride); other overlaps are not
 * allowed.
 * K and the strides are multiples of 8, with q K of 16; K <= 16384 (else
 * MOEQ_ERR_UNSUPPORTED); eps >= 0. */
moeq_status moeq_add_rms_norm(moeq_dtype dtype, const void *x, int64_t x_stride,
                              const void *residual, int64_t residual_stride, int64_t rows,
                              int64_t K, const void *weight, float eps, void *h, void *y,
                              uint8_t *q, float *scales, int32_t row_scales, float *rstd,
                              moeq_stream_t stream);

/* Gradient of moeq_add_rms_norm (of x and of the residual alike; the quantization's is
 * that of v, d_y).  With u = rstd, g = weight * d_y and d_h the gradient that reaches h
 * by itself, along the residual stream:
 *   d_x = u * (g - h * u^2 * mean(g * h)) + d_h;  d_weight = sum over the rows of d_y * h * u
 * fp32; d_weight's sums run in an order that the sizes alone give.
 *   d_y, d_h, h dtype [rows, K], rows strided; d_h NULL: none.
 *   rstd        fp32 [rows], from the forward call.
 *   d_x         dtype [rows, K] (out; may be d_y's, d_h's or h's own buffer, at stride K).
 *   d_weight    fp32 [K] (out) or NULL.  With it, workspace: device memory of
 *               moeq_add_rms_norm_grad_workspace(rows, K) bytes that no other call in
 *               flight uses (two captured graphs that share one do not run at once).
 * rows == 0: d_weight is 0. */
moeq_status moeq_add_rms_norm_grad(moeq_dtype dtype, const void *d_y, int64_t d_y_stride,
                                   const void *d_h, int64_t d_h_stride, const void *h,
                                   int64_t h_stride, int64_t rows, int64_t K, const void *weight,
                                   const float *rstd, void *d_x, float *d_weight, void *workspace,
                                   moeq_stream_t stream);

/* Bytes of that workspace (-1: sizes that the call refuses).  Host only. */
int64_t moeq_add_rms_norm_grad_workspace(int64_t rows, int64_t K);

/* Grouped FP8 matmul with a scale for each block of 128:
 *   c[t, n] = bf16( sum over kb of (a_scales[t, kb] * b_scales[e, n / 128, kb])
 *                   * sum over k in block kb of a[t, k] * b[e, n, k] ),  e = expert_ids[g]
 * the inner sums fp32 on the tensor cores, the outer one fp32 in the order of kb,
 * rounded once.
 *   c         bf16 [total_tokens, N]
 *   a         E4M3 [total_tokens, K];  a_scales fp32 [total_tokens, ceil(K / 128)]
 *   b         E4M3 [num_experts, N, K];  b_scales fp32 [num_experts, ceil(N / 128), ceil(K / 128)]
 * The product of the two scales is rounded to fp32 first: below 2^-126 it loses bits, and
 * from 2^128 on it is infinite (NaN times a zero sum) though the term may not be.
 * K % 16 == 0, N % 8 == 0.  The activations' gradient is the same call on the
 * transposed weights: b [num_experts, K, N] and b_scales [num_experts, ceil(K / 128),
 * ceil(N / 128)] are the same codes and scales with their last two axes exchanged
 * (the caller's copy), a and a_scales the quantized gradient of c, and N is the
 * reduction (N % 16 == 0, K % 8 == 0). */
moeq_status moeq_grouped_matmul_fp8_block(void *c, const uint8_t *a, const uint8_t *b,
                                          const float *a_scales, const float *b_scales,
                                          const uint32_t *a_offsets, const int32_t *expert_ids,
                                          int64_t total_tokens, int64_t N, int64_t K,
                                          int32_t num_experts, int32_t max_tokens_per_expert,
                                          int32_t num_active_experts, moeq_stream_t stream);

/* The same product with an epilogue:
 *   z[t, n] = sum (as above, fp32) + bias[e, n],  c[t, n] = bf16(act(z) + residual[t, n])
 * fp32 up to the one rounding, act one of
 *   relu max(z, 0);  silu z sigma(z);  gelu z Phi(z), Phi the normal distribution within
 *   2^-23;  gelu_tanh z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3)))
 *   bias        fp32 [num_experts, N] or NULL.
 *   residual    bf16 [total_tokens, N] or NULL; may be c itself.
 *   z           bf16 [total_tokens, N] (out) or NULL: z rounded, for the gradient; c is
 *               computed from fp32 z.  No other output or input of the call.
 * Rows outside the groups are not written.  One group of all rows and one expert make it a
 * plain product; the other arguments are as above. */
typedef enum {
    MOEQ_ACT_NONE = 0,
    MOEQ_ACT_RELU = 1,
    MOEQ_ACT_SILU = 2,
    MOEQ_ACT_GELU = 3,
    MOEQ_ACT_GELU_TANH = 4
} moeq_activation;
moeq_status moeq_grouped_matmul_fp8_block_epilogue(
    void *c, const uint8_t *a, const uint8_t *b, const float *a_scales, const float *b_scales,
    const float *bias, moeq_activation activation, const void *residual, void *z,
    const uint32_t *a_offsets, const int32_t *expert_ids, int64_t total_tokens, int64_t N,
    int64_t K, int32_t num_experts, int32_t max_tokens_per_expert, int32_t num_active_experts,
    moeq_stream_t stream);

/* Gradient of that epilogue, from d_c and the saved z:
 *   d_z = d_c * act'(z);  d_bias[e] = sum over the rows of e's groups of d_z
 * fp32; d_z leaves as E4M3 codes q with a scale per 1 x 128 block (the rule of
 * moeq_quantize_fp8_block, from fp32; the operand of the activations' gradient, above) and
 * / or as bf16 d_z (for the weights'); the residual's gradient is d_c itself.  The bias's
 * sums run in an order that the groups give: the same bits every time.
 *   d_c         bf16 [total_tokens, N], row stride d_c_stride elements (a multiple of 8).
 *   z           bf16 [total_tokens, N]; NULL with MOEQ_ACT_NONE and only then.
 *   q           E4M3 [total_tokens, N] (out) and scales fp32 [total_tokens,
 *               ceil(N / 128)] (out), or both NULL;  d_z bf16 [total_tokens, N] (out) or NULL.
 *   d_bias      fp32 [num_experts, N] (out) or NULL; an expert without rows gets 0.  With
 *               it, workspace: device memory of moeq_grouped_epilogue_grad_workspace(...)
 *               bytes that no other call in flight uses.
 * A NaN z makes its d_z NaN, an infinite one too but for relu; an infinity among d_z
 * gives its block an infinite scale and itself a NaN code.
 * Rows outside the groups are not written and not summed; no output overlaps an input or
 * another output.  N % 8 == 0, with q N % 16 == 0;
 * num_experts <= 65535 (else MOEQ_ERR_UNSUPPORTED). */
moeq_status moeq_grouped_epilogue_grad(const void *d_c, int64_t d_c_stride, const void *z,
                                       moeq_activation activation, uint8_t *q, float *scales,
                                       void *d_z, float *d_bias, const uint32_t *a_offsets,
                                       const int32_t *expert_ids, int64_t total_tokens, int64_t N,
                                       int32_t num_experts, int32_t num_active_experts,
                                       void *workspace, moeq_stream_t stream);

/* Bytes of that workspace (-1: sizes that the call refuses).  Host only. */
int64_t moeq_grouped_epilogue_grad_workspace(int64_t total_tokens, int64_t N,
                                             int32_t num_active_experts);

/* Reads the sticky device error word of the current device (MOEQ_DEVERR_*
 * bits) after synchronising `stream`.  Returns MOEQ_ERR_DEVICE when any bit
 * is set, MOEQ_OK otherwise. */
moeq_status moeq_get_device_error(moeq_stream_t stream, uint32_t *bits);

/* Clears the device error word of the current device (enqueued on stream). */
moeq_status moeq_clear_device_error(moeq_stream_t stream);

/* The cudaError_t of the last MOEQ_ERR_CUDA on this thread (0 if none). */
int moeq_last_cuda_error(void);

/* Static string naming a status. */
const char *moeq_status_string(moeq_status s);

#ifdef __cplusplus
}
#endif

#endif /* MOEQ_H */
