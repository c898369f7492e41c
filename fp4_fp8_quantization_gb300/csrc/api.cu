// C ABI of the moeq library: host-side argument validation, the device
// error word, and dispatch to the kernel launchers.  Every compute entry
// point only enqueues work on the caller's stream.
#include <stdint.h>

#include "../../include/moeq.h"
#include "common.cuh"
#include "launch.h"

namespace {

__device__ uint32_t g_device_error;

thread_local int t_last_cuda_error = 0;

// Address of the device error word on the current device (looked up once
// per device).
uint32_t *device_error_ptr() {
    static std::atomic<uint32_t *> cache[moeq::kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= moeq::kMaxDevices) return nullptr;
    return moeq::cached_per_device(cache, dev, []() -> uint32_t * {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
        return static_cast<uint32_t *>(p);
    });
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

moeq_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return MOEQ_OK;
    if (e == cudaErrorNotSupported) return MOEQ_ERR_UNSUPPORTED;
    t_last_cuda_error = (int)e;
    return MOEQ_ERR_CUDA;
}

// Common checks of the ragged-group description.
bool groups_ok(const uint32_t *offs, const int32_t *ids, int32_t num_experts,
               int32_t num_active_experts) {
    if (num_active_experts < 0 || num_experts <= 0) return false;
    if (num_active_experts > 0 && (!offs || !ids)) return false;
    return true;
}

moeq::GroupArgs make_groups(const uint32_t *ro, const uint32_t *so, const int32_t *ids,
                            int32_t G, int32_t E, int64_t rows, int64_t scale_rows) {
    moeq::GroupArgs g;
    g.row_offsets = ro;
    g.scales_offsets = so;
    g.expert_ids = ids;
    g.num_groups = G;
    g.num_experts = E;
    g.total_rows = rows;
    g.scale_rows_total = scale_rows;
    return g;
}

}  // namespace

std::mutex &moeq::launch_setup_mutex() {
    static std::mutex m;
    return m;
}

extern "C" {

const char *moeq_status_string(moeq_status s) {
    switch (s) {
        case MOEQ_OK: return "MOEQ_OK";
        case MOEQ_ERR_INVALID_ARG: return "MOEQ_ERR_INVALID_ARG";
        case MOEQ_ERR_UNSUPPORTED: return "MOEQ_ERR_UNSUPPORTED";
        case MOEQ_ERR_CUDA: return "MOEQ_ERR_CUDA";
        case MOEQ_ERR_DEVICE: return "MOEQ_ERR_DEVICE";
    }
    return "MOEQ_UNKNOWN_STATUS";
}

int moeq_last_cuda_error(void) { return t_last_cuda_error; }

moeq_status moeq_get_device_error(moeq_stream_t stream, uint32_t *bits) {
    if (!bits) return MOEQ_ERR_INVALID_ARG;
    uint32_t *p = device_error_ptr();
    if (!p) return cuda_status(cudaErrorInvalidDevice);
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyAsync(&v, p, sizeof(v), cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_status(e);
    *bits = v;
    return v ? MOEQ_ERR_DEVICE : MOEQ_OK;
}

moeq_status moeq_clear_device_error(moeq_stream_t stream) {
    uint32_t *p = device_error_ptr();
    if (!p) return cuda_status(cudaErrorInvalidDevice);
    return cuda_status(cudaMemsetAsync(p, 0, sizeof(uint32_t), stream));
}

moeq_status moeq_padded_scale_offsets(const uint32_t *row_offsets, uint32_t *scales_offsets,
                                      int32_t num_active_experts, moeq_stream_t stream) {
    if (num_active_experts < 0 || !row_offsets || !scales_offsets) return MOEQ_ERR_INVALID_ARG;
    return cuda_status(
        moeq::launch_padded_offsets(row_offsets, scales_offsets, num_active_experts, stream));
}

// Sizes of the layout helpers: products stay far below 2^62.
static bool layout_sizes_ok(int64_t batch, int64_t rows, int64_t cols) {
    const int64_t lim = (int64_t)1 << 40;
    return batch >= 0 && rows >= 0 && cols >= 0 && batch < lim && rows < lim && cols < lim &&
           (batch == 0 || rows == 0 || cols == 0 ||
            (double)batch * (double)(rows + 128) * (double)(cols + 4) < 4e18);
}

moeq_status moeq_sf_swizzle(uint8_t *tiled, const uint8_t *logical, int64_t batch, int64_t rows,
                            int64_t kv, moeq_stream_t stream) {
    if (!layout_sizes_ok(batch, rows, kv)) return MOEQ_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0 || kv == 0) return MOEQ_OK;
    if (!tiled || !logical) return MOEQ_ERR_INVALID_ARG;
    return cuda_status(moeq::launch_sf_swizzle(tiled, logical, batch, rows, kv, stream));
}

moeq_status moeq_sf_unswizzle(uint8_t *logical, const uint8_t *tiled, int64_t batch,
                              int64_t rows, int64_t kv, moeq_stream_t stream) {
    if (!layout_sizes_ok(batch, rows, kv)) return MOEQ_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0 || kv == 0) return MOEQ_OK;
    if (!tiled || !logical) return MOEQ_ERR_INVALID_ARG;
    return cuda_status(moeq::launch_sf_unswizzle(logical, tiled, batch, rows, kv, stream));
}

moeq_status moeq_interleave_gate_up(uint8_t *out, const uint8_t *gate, const uint8_t *up,
                                    int64_t batch, int64_t rows, int64_t row_bytes,
                                    moeq_stream_t stream) {
    if (!layout_sizes_ok(batch, 2 * rows, row_bytes)) return MOEQ_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0 || row_bytes == 0) return MOEQ_OK;
    if (!out || !gate || !up) return MOEQ_ERR_INVALID_ARG;
    return cuda_status(
        moeq::launch_interleave_rows(out, gate, up, batch, rows, row_bytes, stream));
}

static moeq_status amax_impl(const void *in, int64_t in_row_stride, int64_t total_rows,
                             int64_t K, const uint32_t *row_offsets, const int32_t *expert_ids,
                             float *tensor_scale_out, int32_t num_experts,
                             int32_t num_active_experts, const moeq::Gather &gt,
                             moeq_stream_t stream) {
    if (!groups_ok(row_offsets, expert_ids, num_experts, num_active_experts))
        return MOEQ_ERR_INVALID_ARG;
    if (!tensor_scale_out || total_rows < 0 || K <= 0 || K % 8 || in_row_stride < K ||
        in_row_stride % 8)
        return MOEQ_ERR_INVALID_ARG;
    if (total_rows > 0 && (!in || !aligned16(in))) return MOEQ_ERR_INVALID_ARG;
    if (!aligned16(tensor_scale_out)) return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    moeq::GroupArgs g = make_groups(row_offsets, nullptr, expert_ids, num_active_experts,
                                    num_experts, num_active_experts ? total_rows : 0, 0);
    return cuda_status(
        moeq::launch_amax_scale(in, in_row_stride, K, g, gt, tensor_scale_out, err, stream));
}

static moeq_status quantize_impl(moeq_format fmt, const void *in, int64_t in_row_stride,
                                 int64_t total_rows, int64_t K, uint8_t *out, uint8_t *scales,
                                 int64_t scale_rows_total, const uint32_t *row_offsets,
                                 const uint32_t *scales_offsets, const int32_t *expert_ids,
                                 const float *tensor_scale, int32_t num_experts,
                                 int32_t num_active_experts, const moeq::Gather &gt,
                                 moeq_stream_t stream) {
    if (fmt != MOEQ_NVFP4 && fmt != MOEQ_MXFP4 && fmt != MOEQ_MXFP8) return MOEQ_ERR_INVALID_ARG;
    if (!groups_ok(row_offsets, expert_ids, num_experts, num_active_experts))
        return MOEQ_ERR_INVALID_ARG;
    if (total_rows < 0 || K <= 0 || K % 128 || in_row_stride < K || in_row_stride % 8 ||
        scale_rows_total < 0 || scale_rows_total % 128)
        return MOEQ_ERR_INVALID_ARG;
    if (fmt == MOEQ_NVFP4 && !tensor_scale) return MOEQ_ERR_INVALID_ARG;
    if (num_active_experts == 0 || total_rows == 0 || scale_rows_total == 0) return MOEQ_OK;
    if (!scales_offsets || !in || !out || !scales || !aligned16(in) || !aligned16(out) ||
        !aligned16(scales))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    moeq::GroupArgs g = make_groups(row_offsets, scales_offsets, expert_ids, num_active_experts,
                                    num_experts, total_rows, scale_rows_total);
    return cuda_status(moeq::launch_quantize((int)fmt, in, in_row_stride, K, out, scales,
                                             tensor_scale, g, gt, err, stream));
}

static bool gather_ok(const int32_t *indices, int32_t indices_divisor, int64_t in_rows,
                      int64_t total_rows) {
    return indices_divisor >= 1 && in_rows >= 0 && (total_rows == 0 || indices);
}

moeq_status moeq_grouped_amax_scale(const void *in, int64_t in_row_stride, int64_t total_rows,
                                    int64_t K, const uint32_t *row_offsets,
                                    const int32_t *expert_ids, float *tensor_scale_out,
                                    int32_t num_experts, int32_t num_active_experts,
                                    moeq_stream_t stream) {
    const moeq::Gather none{nullptr, 1, total_rows};
    return amax_impl(in, in_row_stride, total_rows, K, row_offsets, expert_ids, tensor_scale_out,
                     num_experts, num_active_experts, none, stream);
}

moeq_status moeq_grouped_amax_scale_gather(const void *in, int64_t in_row_stride,
                                           int64_t in_rows, int64_t K,
                                           const int32_t *indices, int32_t indices_divisor,
                                           int64_t total_rows, const uint32_t *row_offsets,
                                           const int32_t *expert_ids, float *tensor_scale_out,
                                           int32_t num_experts, int32_t num_active_experts,
                                           moeq_stream_t stream) {
    if (!gather_ok(indices, indices_divisor, in_rows, total_rows)) return MOEQ_ERR_INVALID_ARG;
    if (in_rows == 0 && total_rows > 0 && num_active_experts > 0) return MOEQ_ERR_INVALID_ARG;
    const moeq::Gather gt{indices, indices_divisor, in_rows};
    return amax_impl(in, in_row_stride, total_rows, K, row_offsets, expert_ids, tensor_scale_out,
                     num_experts, num_active_experts, gt, stream);
}

moeq_status moeq_grouped_quantize(moeq_format fmt, const void *in, int64_t in_row_stride,
                                  int64_t total_rows, int64_t K, uint8_t *out, uint8_t *scales,
                                  int64_t scale_rows_total, const uint32_t *row_offsets,
                                  const uint32_t *scales_offsets, const int32_t *expert_ids,
                                  const float *tensor_scale, int32_t num_experts,
                                  int32_t max_tokens_per_expert, int32_t num_active_experts,
                                  moeq_stream_t stream) {
    (void)max_tokens_per_expert;
    const moeq::Gather none{nullptr, 1, total_rows};
    return quantize_impl(fmt, in, in_row_stride, total_rows, K, out, scales, scale_rows_total,
                         row_offsets, scales_offsets, expert_ids, tensor_scale, num_experts,
                         num_active_experts, none, stream);
}

moeq_status moeq_grouped_quantize_gather(moeq_format fmt, const void *in, int64_t in_row_stride,
                                         int64_t in_rows, int64_t K, const int32_t *indices,
                                         int32_t indices_divisor, int64_t total_rows,
                                         uint8_t *out, uint8_t *scales, int64_t scale_rows_total,
                                         const uint32_t *row_offsets,
                                         const uint32_t *scales_offsets,
                                         const int32_t *expert_ids, const float *tensor_scale,
                                         int32_t num_experts, int32_t max_tokens_per_expert,
                                         int32_t num_active_experts, moeq_stream_t stream) {
    (void)max_tokens_per_expert;
    if (!gather_ok(indices, indices_divisor, in_rows, total_rows)) return MOEQ_ERR_INVALID_ARG;
    if (in_rows == 0 && total_rows > 0 && num_active_experts > 0) return MOEQ_ERR_INVALID_ARG;
    const moeq::Gather gt{indices, indices_divisor, in_rows};
    return quantize_impl(fmt, in, in_row_stride, total_rows, K, out, scales, scale_rows_total,
                         row_offsets, scales_offsets, expert_ids, tensor_scale, num_experts,
                         num_active_experts, gt, stream);
}

// ------------------------------------------------------------ dispatch

static moeq_status route_args_ok(const int32_t *topk_ids, int64_t num_tokens, int32_t top_k,
                                 int32_t num_experts, const uint32_t *row_offsets,
                                 const int32_t *expert_ids, const int32_t *src_info,
                                 const int32_t *dst_info, const uint32_t *scales_offsets,
                                 int32_t slot_rows) {
    if (num_tokens < 0 || top_k < 1 || num_experts < 1 || slot_rows < 0 || slot_rows % 128)
        return MOEQ_ERR_INVALID_ARG;
    if (num_experts > moeq::kRouteMaxExperts || num_tokens >= ((int64_t)1 << 31) / top_k)
        return MOEQ_ERR_UNSUPPORTED;
    if (!row_offsets || !expert_ids || !aligned16(row_offsets) || !aligned16(expert_ids))
        return MOEQ_ERR_INVALID_ARG;
    if (scales_offsets && !aligned16(scales_offsets)) return MOEQ_ERR_INVALID_ARG;
    if (dst_info && !aligned16(dst_info)) return MOEQ_ERR_INVALID_ARG;
    if (num_tokens > 0 &&
        (!topk_ids || !src_info || !aligned16(topk_ids) || !aligned16(src_info)))
        return MOEQ_ERR_INVALID_ARG;
    return MOEQ_OK;
}

moeq_status moeq_route_topk(const int32_t *topk_ids, int64_t num_tokens, int32_t top_k,
                            int32_t num_experts, uint32_t *row_offsets, int32_t *expert_ids,
                            int32_t *src_info, int32_t *dst_info, uint32_t *scales_offsets,
                            int32_t slot_rows, moeq_stream_t stream) {
    const moeq_status st = route_args_ok(topk_ids, num_tokens, top_k, num_experts, row_offsets,
                                         expert_ids, src_info, dst_info, scales_offsets,
                                         slot_rows);
    if (st != MOEQ_OK) return st;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    return cuda_status(moeq::launch_route_topk(topk_ids, num_tokens * top_k, num_experts,
                                               row_offsets, expert_ids, src_info, dst_info,
                                               scales_offsets, slot_rows, err, stream));
}

moeq_status moeq_grouped_amax_scale_topk(const void *tokens, int64_t token_stride,
                                         int64_t num_tokens, int64_t K, const int32_t *topk_ids,
                                         int32_t top_k, float *tensor_scale_out,
                                         int32_t num_experts, moeq_stream_t stream) {
    if (num_tokens < 0 || top_k < 1 || num_experts < 1 || K <= 0 || K % 8 ||
        token_stride < K || token_stride % 8 || !tensor_scale_out ||
        !aligned16(tensor_scale_out))
        return MOEQ_ERR_INVALID_ARG;
    if (num_tokens >= ((int64_t)1 << 31) / top_k) return MOEQ_ERR_UNSUPPORTED;
    if (num_tokens > 0 &&
        (!tokens || !topk_ids || !aligned16(tokens) || !aligned16(topk_ids)))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    return cuda_status(moeq::launch_amax_scale_topk(tokens, token_stride, K, num_tokens, topk_ids,
                                                    top_k, num_experts, tensor_scale_out, err,
                                                    stream));
}

int64_t moeq_dispatch_scale_rows(int64_t num_tokens, int32_t top_k, int32_t num_experts,
                                 int32_t slot_rows) {
    if (num_tokens < 0 || top_k < 1 || num_experts < 1 || slot_rows < 0 ||
        num_tokens >= ((int64_t)1 << 31) / top_k)
        return -1;
    if (slot_rows > 0) return (int64_t)num_experts * slot_rows;
    // sum over experts of ceil(r_e / 128) * 128 <= sum (r_e + 127), a multiple of 128
    return (num_tokens * top_k + 127 * (int64_t)num_experts) / 128 * 128;
}

moeq_status moeq_quantize_topk(moeq_format fmt, const void *tokens, int64_t token_stride,
                               int64_t num_tokens, int64_t K, const int32_t *topk_ids,
                               int32_t top_k, const int32_t *dst_info,
                               const uint32_t *row_offsets, const uint32_t *scales_offsets,
                               const float *tensor_scale, int32_t num_experts, uint8_t *out,
                               uint8_t *scales, int64_t scale_rows_total, moeq_stream_t stream) {
    if (fmt != MOEQ_NVFP4 && fmt != MOEQ_MXFP4 && fmt != MOEQ_MXFP8) return MOEQ_ERR_INVALID_ARG;
    if (num_tokens < 0 || top_k < 1 || num_experts < 1 || K <= 0 || K % 128 ||
        token_stride < K || token_stride % 8 || scale_rows_total < 0 || scale_rows_total % 128)
        return MOEQ_ERR_INVALID_ARG;
    if (top_k > moeq::kTopkQuantMax || num_experts > moeq::kRouteMaxExperts ||
        num_tokens >= ((int64_t)1 << 31) / top_k)
        return MOEQ_ERR_UNSUPPORTED;
    if (fmt == MOEQ_NVFP4 && !tensor_scale) return MOEQ_ERR_INVALID_ARG;
    if (!row_offsets || !scales_offsets || !scales || !aligned16(scales)) return MOEQ_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!tokens || !topk_ids || !dst_info || !out || !aligned16(tokens) ||
                           !aligned16(topk_ids) || !aligned16(dst_info) || !aligned16(out)))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    return cuda_status(moeq::launch_quantize_topk(
        (int)fmt, tokens, token_stride, K, num_tokens, topk_ids, top_k, dst_info, row_offsets,
        scales_offsets, tensor_scale, num_experts, num_tokens * top_k, scale_rows_total, out,
        scales, err, stream));
}

moeq_status moeq_dispatch_mxfp4(const void *tokens, int64_t token_stride, int64_t num_tokens,
                                int64_t hidden, const int32_t *topk_ids, int32_t top_k,
                                int32_t num_experts, uint8_t *out, uint8_t *scales,
                                int64_t scale_rows_total, uint32_t *row_offsets,
                                int32_t *expert_ids, int32_t *src_info, int32_t *dst_info,
                                uint32_t *scales_offsets, int32_t slot_rows,
                                moeq_stream_t stream) {
    moeq_status st = route_args_ok(topk_ids, num_tokens, top_k, num_experts, row_offsets,
                                   expert_ids, src_info, dst_info, scales_offsets, slot_rows);
    if (st != MOEQ_OK) return st;
    // every check of the quantization step before anything is launched
    if (!scales_offsets || hidden <= 0 || hidden % 128 || token_stride < hidden ||
        token_stride % 8 || scale_rows_total % 128 || !scales || !aligned16(scales) ||
        scale_rows_total < moeq_dispatch_scale_rows(num_tokens, top_k, num_experts, slot_rows))
        return MOEQ_ERR_INVALID_ARG;
    if (top_k > moeq::kTopkQuantMax) return MOEQ_ERR_UNSUPPORTED;
    if (num_tokens > 0 && (!tokens || !out || !dst_info || !aligned16(tokens) || !aligned16(out)))
        return MOEQ_ERR_INVALID_ARG;
    st = moeq_route_topk(topk_ids, num_tokens, top_k, num_experts, row_offsets, expert_ids,
                         src_info, dst_info, scales_offsets, slot_rows, stream);
    if (st != MOEQ_OK) return st;
    // token-major: each token read and quantized once, stored to its routed rows
    return moeq_quantize_topk(MOEQ_MXFP4, tokens, token_stride, num_tokens, hidden, topk_ids,
                              top_k, dst_info, row_offsets, scales_offsets, nullptr, num_experts,
                              out, scales, scale_rows_total, stream);
}

moeq_status moeq_grouped_matmul_rowwise_fp8(void *c, const uint8_t *a, const uint8_t *b,
                                            const float *a_scales, const float *b_scales,
                                            const uint32_t *a_offsets,
                                            const int32_t *expert_ids, int64_t total_tokens,
                                            int64_t N, int64_t K, int32_t num_experts,
                                            int32_t max_tokens_per_expert,
                                            int32_t num_active_experts, moeq_stream_t stream) {
    if (!groups_ok(a_offsets, expert_ids, num_experts, num_active_experts))
        return MOEQ_ERR_INVALID_ARG;
    if (total_tokens < 0 || N <= 0 || K <= 0 || K % 128 || N % 16) return MOEQ_ERR_INVALID_ARG;
    if (total_tokens >= (int64_t)1 << 31 || N >= (int64_t)1 << 31 || K >= (int64_t)1 << 31)
        return MOEQ_ERR_UNSUPPORTED;
    if (num_active_experts > moeq::kMaxGroups) return MOEQ_ERR_UNSUPPORTED;
    if (!b || !b_scales || !aligned16(b) || !aligned16(b_scales)) return MOEQ_ERR_INVALID_ARG;
    if (num_active_experts == 0 || total_tokens == 0) return MOEQ_OK;
    if (!c || !a || !a_scales || !aligned16(c) || !aligned16(a) || !aligned16(a_scales))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    moeq::GemmArgs ga = {};
    ga.kind = 0;
    ga.epi = 0;
    ga.groups = make_groups(a_offsets, nullptr, expert_ids, num_active_experts, num_experts,
                            total_tokens, 0);
    ga.N = N;
    ga.K = K;
    ga.a = a;
    ga.b = b;
    ga.a_scales = a_scales;
    ga.b_scales = b_scales;
    ga.c = c;
    ga.max_tokens_per_expert = max_tokens_per_expert;
    ga.err = err;
    return cuda_status(moeq::launch_gemm(ga, stream));
}

static moeq_status blockscaled_common(moeq_format fmt, int epi, const uint8_t *a,
                                      const uint8_t *a_sf, const uint8_t *b, const uint8_t *b_sf,
                                      const uint32_t *a_offsets,
                                      const uint32_t *a_scales_offsets,
                                      const int32_t *expert_ids, int64_t total_tokens,
                                      int64_t scale_rows_total, int64_t N, int64_t K,
                                      int32_t num_experts, int32_t num_active_experts,
                                      moeq::GemmArgs *ga) {
    if (!groups_ok(a_offsets, expert_ids, num_experts, num_active_experts))
        return MOEQ_ERR_INVALID_ARG;
    if (fmt != MOEQ_NVFP4 && fmt != MOEQ_MXFP4 && fmt != MOEQ_MXFP8) return MOEQ_ERR_INVALID_ARG;
    if (total_tokens < 0 || N <= 0 || K <= 0 || N % 128 || scale_rows_total < 0 ||
        scale_rows_total % 128)
        return MOEQ_ERR_INVALID_ARG;
    if (fmt == MOEQ_MXFP8 ? (K % 128) : (K % 256)) return MOEQ_ERR_INVALID_ARG;
    if (total_tokens >= (int64_t)1 << 31 || N >= (int64_t)1 << 31 || K >= (int64_t)1 << 31)
        return MOEQ_ERR_UNSUPPORTED;
    if (num_active_experts > moeq::kMaxGroups) return MOEQ_ERR_UNSUPPORTED;
    if (!b || !b_sf || !aligned16(b) || !aligned16(b_sf)) return MOEQ_ERR_INVALID_ARG;
    if (num_active_experts > 0 && !a_scales_offsets) return MOEQ_ERR_INVALID_ARG;
    if (num_active_experts > 0 && total_tokens > 0 &&
        (!a || !a_sf || !aligned16(a) || !aligned16(a_sf)))
        return MOEQ_ERR_INVALID_ARG;
    *ga = moeq::GemmArgs{};
    ga->kind = fmt == MOEQ_NVFP4 ? 1 : (fmt == MOEQ_MXFP8 ? 2 : 3);
    ga->epi = epi;
    ga->groups = make_groups(a_offsets, a_scales_offsets, expert_ids, num_active_experts,
                             num_experts, total_tokens, scale_rows_total);
    ga->N = N;
    ga->K = K;
    ga->a = a;
    ga->b = b;
    ga->a_sf = a_sf;
    ga->b_sf = b_sf;
    return MOEQ_OK;
}

moeq_status moeq_grouped_matmul_blockscaled(
    moeq_format fmt, void *c, const uint8_t *a, const uint8_t *a_sf, const uint8_t *b,
    const uint8_t *b_sf, const float *expert_scales, const uint32_t *a_offsets,
    const uint32_t *a_scales_offsets, const int32_t *expert_ids, int64_t total_tokens,
    int64_t scale_rows_total, int64_t N, int64_t K, int32_t num_experts,
    int32_t max_tokens_per_expert, int32_t num_active_experts, moeq_stream_t stream) {
    moeq::GemmArgs ga;
    moeq_status st =
        blockscaled_common(fmt, 0, a, a_sf, b, b_sf, a_offsets, a_scales_offsets, expert_ids,
                           total_tokens, scale_rows_total, N, K, num_experts,
                           num_active_experts, &ga);
    if (st != MOEQ_OK) return st;
    if (fmt == MOEQ_NVFP4 && !expert_scales) return MOEQ_ERR_INVALID_ARG;
    if (expert_scales && !aligned16(expert_scales)) return MOEQ_ERR_INVALID_ARG;
    if (num_active_experts == 0 || total_tokens == 0) return MOEQ_OK;
    if (!c || !aligned16(c)) return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    ga.expert_scales = expert_scales;
    ga.c = c;
    ga.max_tokens_per_expert = max_tokens_per_expert;
    ga.err = err;
    return cuda_status(moeq::launch_gemm(ga, stream));
}

static moeq_status swiglu_quantize_impl(int out_fmt, uint8_t *c_q, uint8_t *c_sf, const void *y,
                                        const float *out_tensor_scale, const uint32_t *a_offsets,
                                        const uint32_t *a_scales_offsets,
                                        const int32_t *expert_ids, int64_t total_tokens,
                                        int64_t scale_rows_total, int64_t I, int32_t num_experts,
                                        int32_t num_active_experts, moeq_stream_t stream) {
    if (!groups_ok(a_offsets, expert_ids, num_experts, num_active_experts))
        return MOEQ_ERR_INVALID_ARG;
    if (total_tokens < 0 || I <= 0 || I % (out_fmt == 0 ? 64 : 128) || scale_rows_total < 0 ||
        scale_rows_total % 128)
        return MOEQ_ERR_INVALID_ARG;
    if (out_fmt == 0 && !out_tensor_scale) return MOEQ_ERR_INVALID_ARG;
    if (num_active_experts == 0 || total_tokens == 0 || scale_rows_total == 0) return MOEQ_OK;
    if (!a_scales_offsets || !y || !c_q || !c_sf || !aligned16(y) || !aligned16(c_q) ||
        !aligned16(c_sf))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    moeq::GroupArgs g = make_groups(a_offsets, a_scales_offsets, expert_ids, num_active_experts,
                                    num_experts, total_tokens, scale_rows_total);
    return cuda_status(moeq::launch_swiglu_quantize(out_fmt, c_q, c_sf, y, I, out_tensor_scale, g,
                                                    err, stream));
}

moeq_status moeq_swiglu_quantize(uint8_t *c_packed, uint8_t *c_sf, const void *y,
                                 const float *out_tensor_scale, const uint32_t *a_offsets,
                                 const uint32_t *a_scales_offsets, const int32_t *expert_ids,
                                 int64_t total_tokens, int64_t scale_rows_total, int64_t I,
                                 int32_t num_experts, int32_t max_tokens_per_expert,
                                 int32_t num_active_experts, moeq_stream_t stream) {
    (void)max_tokens_per_expert;
    return swiglu_quantize_impl(0, c_packed, c_sf, y, out_tensor_scale, a_offsets,
                                a_scales_offsets, expert_ids, total_tokens, scale_rows_total, I,
                                num_experts, num_active_experts, stream);
}

moeq_status moeq_swiglu_quantize_mx(moeq_format fmt, uint8_t *c_q, uint8_t *c_sf, const void *y,
                                    const uint32_t *a_offsets, const uint32_t *a_scales_offsets,
                                    const int32_t *expert_ids, int64_t total_tokens,
                                    int64_t scale_rows_total, int64_t I, int32_t num_experts,
                                    int32_t max_tokens_per_expert, int32_t num_active_experts,
                                    moeq_stream_t stream) {
    (void)max_tokens_per_expert;
    if (fmt != MOEQ_MXFP4 && fmt != MOEQ_MXFP8) return MOEQ_ERR_INVALID_ARG;
    return swiglu_quantize_impl((int)fmt, c_q, c_sf, y, nullptr, a_offsets, a_scales_offsets,
                                expert_ids, total_tokens, scale_rows_total, I, num_experts,
                                num_active_experts, stream);
}

moeq_status moeq_grouped_matmul_swiglu(
    uint8_t *c_packed, uint8_t *c_sf, const uint8_t *a, const uint8_t *a_sf, const uint8_t *b,
    const uint8_t *b_sf, const float *expert_scales, const float *out_tensor_scale,
    const void *a_row_scales, const uint32_t *a_offsets, const uint32_t *a_scales_offsets,
    const int32_t *expert_ids, int64_t total_tokens, int64_t scale_rows_total, int64_t I,
    int64_t K, int32_t num_experts, int32_t max_tokens_per_expert, int32_t num_active_experts,
    moeq_stream_t stream) {
    if (I <= 0 || I % 64) return MOEQ_ERR_INVALID_ARG;
    moeq::GemmArgs ga;
    moeq_status st = blockscaled_common(MOEQ_NVFP4, 1, a, a_sf, b, b_sf, a_offsets,
                                        a_scales_offsets, expert_ids, total_tokens,
                                        scale_rows_total, 2 * I, K, num_experts,
                                        num_active_experts, &ga);
    if (st != MOEQ_OK) return st;
    if (!expert_scales || !out_tensor_scale) return MOEQ_ERR_INVALID_ARG;
    if (a_row_scales && !aligned16(a_row_scales)) return MOEQ_ERR_INVALID_ARG;
    if (num_active_experts == 0 || total_tokens == 0) return MOEQ_OK;
    if (!c_packed || !c_sf || !aligned16(c_packed) || !aligned16(c_sf))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    ga.expert_scales = expert_scales;
    ga.out_tensor_scale = out_tensor_scale;
    ga.row_scales = static_cast<const uint16_t *>(a_row_scales);
    ga.c_packed = c_packed;
    ga.c_sf = c_sf;
    ga.max_tokens_per_expert = max_tokens_per_expert;
    ga.err = err;
    return cuda_status(moeq::launch_gemm(ga, stream));
}

moeq_status moeq_grouped_matmul_swiglu_mx(
    moeq_format fmt, uint8_t *c_q, uint8_t *c_sf, const uint8_t *a, const uint8_t *a_sf,
    const uint8_t *b, const uint8_t *b_sf, const float *expert_scales, const uint32_t *a_offsets,
    const uint32_t *a_scales_offsets, const int32_t *expert_ids, int64_t total_tokens,
    int64_t scale_rows_total, int64_t I, int64_t K, int32_t num_experts,
    int32_t max_tokens_per_expert, int32_t num_active_experts, moeq_stream_t stream) {
    if (fmt != MOEQ_MXFP4 && fmt != MOEQ_MXFP8) return MOEQ_ERR_INVALID_ARG;
    if (I <= 0 || I % 128) return MOEQ_ERR_INVALID_ARG;
    moeq::GemmArgs ga;
    moeq_status st = blockscaled_common(fmt, 2, a, a_sf, b, b_sf, a_offsets, a_scales_offsets,
                                        expert_ids, total_tokens, scale_rows_total, 2 * I, K,
                                        num_experts, num_active_experts, &ga);
    if (st != MOEQ_OK) return st;
    if (expert_scales && !aligned16(expert_scales)) return MOEQ_ERR_INVALID_ARG;
    if (num_active_experts == 0 || total_tokens == 0) return MOEQ_OK;
    if (!c_q || !c_sf || !aligned16(c_q) || !aligned16(c_sf)) return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    ga.expert_scales = expert_scales;
    ga.c_packed = c_q;
    ga.c_sf = c_sf;
    ga.max_tokens_per_expert = max_tokens_per_expert;
    ga.err = err;
    return cuda_status(moeq::launch_gemm(ga, stream));
}

// ------------------------------------------------ router, rows, FP8 blocks

static bool dtype_ok(int dt) { return dt == MOEQ_BF16 || dt == MOEQ_FP16 || dt == MOEQ_FP32; }
static int64_t dtype_size(int dt) { return dt == MOEQ_FP32 ? 4 : 2; }

static moeq_status gate_args_ok(moeq_dtype dt, const void *logits, int64_t stride,
                                int64_t num_tokens, int32_t num_experts, int32_t top_k) {
    if (!dtype_ok(dt) || num_tokens < 0 || num_experts < 1 || top_k < 1 || top_k > num_experts ||
        stride < num_experts)
        return MOEQ_ERR_INVALID_ARG;
    if (num_experts > moeq::kRouteMaxExperts || top_k > moeq::kTopkRowsMax ||
        num_tokens >= ((int64_t)1 << 31) / top_k)
        return MOEQ_ERR_UNSUPPORTED;
    if (num_tokens > 0 && (!logits || !aligned16(logits))) return MOEQ_ERR_INVALID_ARG;
    return MOEQ_OK;
}

moeq_status moeq_gate_topk(moeq_dtype dtype, const void *logits, int64_t logit_stride,
                           int64_t num_tokens, int32_t num_experts, int32_t top_k,
                           int32_t normalize, float scale, int32_t *topk_ids, float *weights,
                           moeq_stream_t stream) {
    const moeq_status st =
        gate_args_ok(dtype, logits, logit_stride, num_tokens, num_experts, top_k);
    if (st != MOEQ_OK) return st;
    if (num_tokens == 0) return MOEQ_OK;
    if (!topk_ids || !weights || !aligned16(topk_ids) || !aligned16(weights))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    moeq::GateArgs a = {};
    a.dtype = dtype;
    a.logits = logits;
    a.stride = logit_stride;
    a.num_tokens = num_tokens;
    a.num_experts = num_experts;
    a.top_k = top_k;
    a.normalize = normalize != 0;
    a.scale = scale;
    a.ids = topk_ids;
    a.weights = weights;
    a.err = err;
    return cuda_status(moeq::launch_gate(a, stream));
}

// chosen: 0 the softmax's gradient over all experts or the choices, 1 that of the
// chosen logits only with sigmoid scores, 2 with softmax scores.
static moeq_status gate_grad_call(moeq_dtype dtype, const void *logits, int64_t logit_stride,
                                  int64_t num_tokens, int32_t num_experts, int32_t top_k,
                                  int32_t normalize, float scale, const int32_t *topk_ids,
                                  const float *d_weights, void *d_logits, int chosen,
                                  moeq_stream_t stream) {
    const moeq_status st =
        gate_args_ok(dtype, logits, logit_stride, num_tokens, num_experts, top_k);
    if (st != MOEQ_OK) return st;
    if (num_tokens == 0) return MOEQ_OK;
    if (!topk_ids || !d_weights || !d_logits || !aligned16(topk_ids) || !aligned16(d_weights) ||
        !aligned16(d_logits) || (chosen && d_logits == logits))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    moeq::GateArgs a = {};
    a.dtype = dtype;
    a.logits = logits;
    a.stride = logit_stride;
    a.num_tokens = num_tokens;
    a.num_experts = num_experts;
    a.top_k = top_k;
    a.normalize = normalize != 0;
    a.scale = scale;
    a.ids = const_cast<int32_t *>(topk_ids);
    a.d_weights = d_weights;
    a.d_logits = d_logits;
    a.err = err;
    return cuda_status(chosen ? moeq::launch_gate_chosen_grad(a, chosen == 1, stream)
                              : moeq::launch_gate(a, stream));
}

moeq_status moeq_gate_topk_grad(moeq_dtype dtype, const void *logits, int64_t logit_stride,
                                int64_t num_tokens, int32_t num_experts, int32_t top_k,
                                int32_t normalize, float scale, const int32_t *topk_ids,
                                const float *d_weights, void *d_logits, moeq_stream_t stream) {
    return gate_grad_call(dtype, logits, logit_stride, num_tokens, num_experts, top_k, normalize,
                          scale, topk_ids, d_weights, d_logits, 0, stream);
}

moeq_status moeq_gate_group_topk_grad(moeq_dtype dtype, const void *logits, int64_t logit_stride,
                                      int64_t num_tokens, int32_t num_experts, moeq_score score,
                                      int32_t top_k, int32_t normalize, float scale,
                                      const int32_t *topk_ids, const float *d_weights,
                                      void *d_logits, moeq_stream_t stream) {
    if (score != MOEQ_SCORE_SOFTMAX && score != MOEQ_SCORE_SIGMOID) return MOEQ_ERR_INVALID_ARG;
    const int chosen = score == MOEQ_SCORE_SIGMOID ? 1 : normalize ? 2 : 0;
    return gate_grad_call(dtype, logits, logit_stride, num_tokens, num_experts, top_k, normalize,
                          scale, topk_ids, d_weights, d_logits, chosen, stream);
}

moeq_status moeq_gate_group_topk(moeq_dtype dtype, const void *logits, int64_t logit_stride,
                                 int64_t num_tokens, int32_t num_experts, const float *bias,
                                 moeq_score score, int32_t num_groups, int32_t topk_groups,
                                 moeq_group_score group_score, int32_t top_k, int32_t normalize,
                                 float scale, int32_t *topk_ids, float *weights,
                                 moeq_stream_t stream) {
    if ((score != MOEQ_SCORE_SOFTMAX && score != MOEQ_SCORE_SIGMOID) ||
        (group_score != MOEQ_GROUP_MAX && group_score != MOEQ_GROUP_TOP2) || num_groups < 1 ||
        topk_groups < 1 || topk_groups > num_groups || num_experts % num_groups)
        return MOEQ_ERR_INVALID_ARG;
    const moeq_status st =
        gate_args_ok(dtype, logits, logit_stride, num_tokens, num_experts, top_k);
    if (st != MOEQ_OK) return st;
    const int32_t size = num_experts / num_groups;
    if (top_k > topk_groups * size) return MOEQ_ERR_INVALID_ARG;
    int32_t lanes = 1;
    while (lanes < num_groups) lanes *= 2;
    if (num_groups > moeq::kMaxExpertGroups || size > 1024 / lanes) return MOEQ_ERR_UNSUPPORTED;
    if (num_tokens == 0) return MOEQ_OK;
    if (!topk_ids || !weights || !aligned16(topk_ids) || !aligned16(weights) || !aligned16(bias))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    const moeq::GateScoredArgs a{(int)dtype, logits, logit_stride, num_tokens, num_experts, top_k,
                                 bias, score == MOEQ_SCORE_SIGMOID,
                                 group_score == MOEQ_GROUP_TOP2, num_groups, topk_groups,
                                 normalize != 0, scale, topk_ids, weights, err};
    return cuda_status(moeq::launch_gate_scored(a, stream));
}

// Common checks of the calls between tokens and their rows.
static moeq_status rows_args_ok(moeq_dtype dt, int64_t token_stride, int64_t num_tokens,
                                int64_t hidden, const int32_t *dst, int32_t top_k,
                                const float *weights, int64_t total_rows) {
    if (!dtype_ok(dt) || num_tokens < 0 || hidden <= 0 || top_k < 1 || total_rows < 0 ||
        token_stride < hidden || hidden * dtype_size(dt) % 16 || token_stride * dtype_size(dt) % 16)
        return MOEQ_ERR_INVALID_ARG;
    if (top_k > moeq::kTopkRowsMax || num_tokens >= ((int64_t)1 << 31) / top_k ||
        total_rows >= (int64_t)1 << 31 || hidden >= (int64_t)1 << 24)
        return MOEQ_ERR_UNSUPPORTED;
    if (num_tokens > 0 && (!dst || !aligned16(dst) || !aligned16(weights)))
        return MOEQ_ERR_INVALID_ARG;
    return MOEQ_OK;
}

static moeq_status rows_call(bool spread, moeq_dtype dtype, const void *token_in,
                             int64_t token_stride, void *token_out, const void *rows_in,
                             void *rows_out, int64_t num_tokens, int64_t hidden,
                             const int32_t *dst, int32_t top_k, const float *weights,
                             float *d_weights, int64_t total_rows, moeq_stream_t stream) {
    const moeq_status st = rows_args_ok(dtype, token_stride, num_tokens, hidden, dst, top_k,
                                        weights, total_rows);
    if (st != MOEQ_OK) return st;
    if (num_tokens == 0) return MOEQ_OK;
    // the token side is always there; the row side may have no rows
    const void *tok = spread ? token_in : token_out, *rows = spread ? rows_out : rows_in;
    if (!tok || !aligned16(tok) || !aligned16(rows) || (total_rows > 0 && !rows))
        return MOEQ_ERR_INVALID_ARG;
    if (d_weights) {
        const void *other = spread ? rows_in : token_in;
        const bool needed = !spread || total_rows > 0;
        if (!aligned16(d_weights) || !aligned16(other) || (needed && !other))
            return MOEQ_ERR_INVALID_ARG;
    }
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    const moeq::RowsArgs a{(int)dtype, spread, token_in, token_stride, token_out, rows_in, rows_out,
                           dst, weights, d_weights, num_tokens, total_rows, hidden, top_k, err};
    return cuda_status(moeq::launch_topk_rows(a, stream));
}

moeq_status moeq_permute_topk(moeq_dtype dtype, const void *tokens, int64_t token_stride,
                              int64_t num_tokens, int64_t hidden, const int32_t *dst_info,
                              int32_t top_k, const float *weights, void *rows, int64_t total_rows,
                              moeq_stream_t stream) {
    return rows_call(true, dtype, tokens, token_stride, nullptr, nullptr, rows, num_tokens, hidden,
                     dst_info, top_k, weights, nullptr, total_rows, stream);
}

moeq_status moeq_permute_topk_grad(moeq_dtype dtype, const void *d_rows, int64_t total_rows,
                                   int64_t num_tokens, int64_t hidden, const int32_t *dst_info,
                                   int32_t top_k, const float *weights, void *d_tokens,
                                   const void *tokens, int64_t token_stride, float *d_weights,
                                   moeq_stream_t stream) {
    return rows_call(false, dtype, tokens, tokens ? token_stride : hidden, d_tokens, d_rows, nullptr,
                     num_tokens, hidden, dst_info, top_k, weights, d_weights, total_rows, stream);
}

moeq_status moeq_combine_topk(moeq_dtype dtype, const void *rows, int64_t total_rows,
                              int64_t num_tokens, int64_t hidden, const int32_t *dst_info,
                              int32_t top_k, const float *weights, void *out,
                              moeq_stream_t stream) {
    return rows_call(false, dtype, nullptr, hidden, out, rows, nullptr, num_tokens, hidden, dst_info,
                     top_k, weights, nullptr, total_rows, stream);
}

moeq_status moeq_combine_topk_grad(moeq_dtype dtype, const void *d_out, int64_t d_out_stride,
                                   int64_t num_tokens, int64_t hidden, const int32_t *dst_info,
                                   int32_t top_k, const float *weights, void *d_rows,
                                   int64_t total_rows, const void *rows, float *d_weights,
                                   moeq_stream_t stream) {
    return rows_call(true, dtype, d_out, d_out_stride, nullptr, rows, d_rows, num_tokens, hidden,
                     dst_info, top_k, weights, d_weights, total_rows, stream);
}

static moeq_status fp8_block_call(const void *in, int64_t stride, int64_t rows, int64_t K,
                                  const int32_t *dst, int32_t top_k, int64_t out_rows, bool swiglu,
                                  uint8_t *out, float *scales, moeq_stream_t stream) {
    if (rows < 0 || K <= 0 || K % 16 || stride < (swiglu ? 2 * K : K) || stride % 8 || out_rows < 0)
        return MOEQ_ERR_INVALID_ARG;
    if (rows >= ((int64_t)1 << 31) / top_k || K >= (int64_t)1 << 31 || out_rows >= (int64_t)1 << 31)
        return MOEQ_ERR_UNSUPPORTED;
    if (rows == 0) return MOEQ_OK;
    if (!in || !aligned16(in) || !aligned16(out) || !aligned16(scales) || (dst && !aligned16(dst)))
        return MOEQ_ERR_INVALID_ARG;
    if (out_rows > 0 && (!out || !scales)) return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    const moeq::Fp8BlockArgs a{in, stride, rows, K, dst, top_k, out_rows, swiglu, out, scales, err};
    return cuda_status(moeq::launch_fp8_block(a, stream));
}

moeq_status moeq_quantize_fp8_block(const void *in, int64_t in_row_stride, int64_t rows, int64_t K,
                                    uint8_t *out, float *scales, moeq_stream_t stream) {
    return fp8_block_call(in, in_row_stride, rows, K, nullptr, 1, rows, false, out, scales, stream);
}

moeq_status moeq_quantize_fp8_block_topk(const void *tokens, int64_t token_stride,
                                         int64_t num_tokens, int64_t K, const int32_t *dst_info,
                                         int32_t top_k, uint8_t *out, float *scales,
                                         int64_t total_rows, moeq_stream_t stream) {
    if (top_k < 1) return MOEQ_ERR_INVALID_ARG;
    if (top_k > moeq::kTopkRowsMax) return MOEQ_ERR_UNSUPPORTED;
    if (num_tokens > 0 && !dst_info) return MOEQ_ERR_INVALID_ARG;
    return fp8_block_call(tokens, token_stride, num_tokens, K, dst_info, top_k, total_rows, false,
                          out, scales, stream);
}

moeq_status moeq_swiglu_quantize_fp8_block(const void *y, int64_t rows, int64_t I, uint8_t *out,
                                           float *scales, moeq_stream_t stream) {
    return fp8_block_call(y, 2 * I, rows, I, nullptr, 1, rows, true, out, scales, stream);
}

moeq_status moeq_quantize_fp8_block_weight(const void *w, int64_t num_experts, int64_t N, int64_t K,
                                           uint8_t *out, float *scales, moeq_stream_t stream) {
    if (num_experts < 0 || N < 0 || K <= 0 || K % 16) return MOEQ_ERR_INVALID_ARG;
    // the launch grid holds one CTA per 128 x 128 block
    if (num_experts > 65535 || (N + 127) / 128 > 65535 || K >= (int64_t)1 << 31)
        return MOEQ_ERR_UNSUPPORTED;
    if (num_experts == 0 || N == 0) return MOEQ_OK;
    if (!w || !out || !scales || !aligned16(w) || !aligned16(out) || !aligned16(scales))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    return cuda_status(
        moeq::launch_fp8_block_weight(w, num_experts, N, K, out, scales, err, stream));
}

static moeq_status norm_sizes_ok(int64_t rows, int64_t K) {
    if (rows < 0 || K <= 0 || K % 8) return MOEQ_ERR_INVALID_ARG;
    if (rows >= (int64_t)1 << 31 || K > moeq::kNormMaxCols) return MOEQ_ERR_UNSUPPORTED;
    return MOEQ_OK;
}

// A strided matrix of 16-byte vectors; one that may be absent.
static bool rows_ok(const void *p, int64_t stride, int64_t K, bool required) {
    return p ? aligned16(p) && stride >= K && stride % 8 == 0 : !required;
}

moeq_status moeq_add_rms_norm(moeq_dtype dtype, const void *x, int64_t x_stride,
                              const void *residual, int64_t residual_stride, int64_t rows,
                              int64_t K, const void *weight, float eps, void *h, void *y,
                              uint8_t *q, float *scales, int32_t row_scales, float *rstd,
                              moeq_stream_t stream) {
    if (!dtype_ok(dtype) || !(eps >= 0.0f)) return MOEQ_ERR_INVALID_ARG;
    const moeq_status st = norm_sizes_ok(rows, K);
    if (st != MOEQ_OK) return st;
    if (rows == 0) return MOEQ_OK;
    if (!rows_ok(x, x_stride, K, true) || !rows_ok(residual, residual_stride, K, false) ||
        !weight || !aligned16(weight) || !aligned16(h) || !aligned16(y) || !aligned16(q) ||
        !aligned16(scales) || !aligned16(rstd))
        return MOEQ_ERR_INVALID_ARG;
    if (!h != !residual || (h && h == y) || !q != !scales || (q && K % 16) || (!y && !q && !rstd))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    const moeq::NormArgs a{(int)dtype, x, residual, weight, x_stride, residual_stride, rows, K,
                           eps, h, y, q, scales, row_scales != 0, rstd, err};
    return cuda_status(moeq::launch_norm(a, stream));
}

int64_t moeq_add_rms_norm_grad_workspace(int64_t rows, int64_t K) {
    if (norm_sizes_ok(rows, K) != MOEQ_OK) return -1;
    return rows ? moeq::norm_grad_parts(rows, K) * K * 4 : 0;
}

moeq_status moeq_add_rms_norm_grad(moeq_dtype dtype, const void *d_y, int64_t d_y_stride,
                                   const void *d_h, int64_t d_h_stride, const void *h,
                                   int64_t h_stride, int64_t rows, int64_t K, const void *weight,
                                   const float *rstd, void *d_x, float *d_weight, void *workspace,
                                   moeq_stream_t stream) {
    if (!dtype_ok(dtype)) return MOEQ_ERR_INVALID_ARG;
    const moeq_status st = norm_sizes_ok(rows, K);
    if (st != MOEQ_OK) return st;
    if (rows == 0 && !d_weight) return MOEQ_OK;
    if (rows > 0 && (!rows_ok(d_y, d_y_stride, K, true) || !rows_ok(d_h, d_h_stride, K, false) ||
        !rows_ok(h, h_stride, K, true) || !weight || !aligned16(weight) || !rstd ||
        !aligned16(rstd) || !d_x || !aligned16(d_x) || (d_weight && !workspace)))
        return MOEQ_ERR_INVALID_ARG;
    if (!aligned16(d_weight) || !aligned16(workspace)) return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    const moeq::NormGradArgs a{(int)dtype, d_y, d_h, h, weight, d_y_stride, d_h_stride, h_stride,
                               rows, K, rstd, d_x, d_weight, static_cast<float *>(workspace), err};
    return cuda_status(moeq::launch_norm_grad(a, stream));
}

static moeq_status matmul_fp8_block_call(moeq::GemmBlockArgs ga, const uint32_t *a_offsets,
                                         const int32_t *expert_ids, int64_t total_tokens,
                                         int32_t num_experts, int32_t num_active_experts,
                                         moeq_stream_t stream) {
    const int64_t N = ga.N, K = ga.K;
    if (!groups_ok(a_offsets, expert_ids, num_experts, num_active_experts))
        return MOEQ_ERR_INVALID_ARG;
    if (total_tokens < 0 || N <= 0 || K <= 0 || K % 16 || N % 8) return MOEQ_ERR_INVALID_ARG;
    if (total_tokens >= (int64_t)1 << 31 || N >= (int64_t)1 << 31 || K >= (int64_t)1 << 31 ||
        num_active_experts > moeq::kMaxGroups)
        return MOEQ_ERR_UNSUPPORTED;
    if (!ga.b || !ga.b_scales || !aligned16(ga.b) || !aligned16(ga.b_scales) ||
        !aligned16(ga.bias))
        return MOEQ_ERR_INVALID_ARG;
    if (num_active_experts == 0 || total_tokens == 0) return MOEQ_OK;
    if (!ga.c || !ga.a || !ga.a_scales || !aligned16(ga.c) || !aligned16(ga.a) ||
        !aligned16(ga.a_scales) || !aligned16(ga.residual) || !aligned16(ga.z))
        return MOEQ_ERR_INVALID_ARG;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    ga.groups = make_groups(a_offsets, nullptr, expert_ids, num_active_experts, num_experts,
                            total_tokens, 0);
    ga.err = err;
    return cuda_status(moeq::launch_gemm_fp8_block(ga, stream));
}

moeq_status moeq_grouped_matmul_fp8_block(void *c, const uint8_t *a, const uint8_t *b,
                                          const float *a_scales, const float *b_scales,
                                          const uint32_t *a_offsets, const int32_t *expert_ids,
                                          int64_t total_tokens, int64_t N, int64_t K,
                                          int32_t num_experts, int32_t max_tokens_per_expert,
                                          int32_t num_active_experts, moeq_stream_t stream) {
    (void)max_tokens_per_expert;
    moeq::GemmBlockArgs ga = {};
    ga.N = N;
    ga.K = K;
    ga.a = a;
    ga.b = b;
    ga.a_scales = a_scales;
    ga.b_scales = b_scales;
    ga.c = c;
    return matmul_fp8_block_call(ga, a_offsets, expert_ids, total_tokens, num_experts,
                                 num_active_experts, stream);
}

static bool activation_ok(int act) { return act >= MOEQ_ACT_NONE && act <= MOEQ_ACT_GELU_TANH; }

moeq_status moeq_grouped_matmul_fp8_block_epilogue(
    void *c, const uint8_t *a, const uint8_t *b, const float *a_scales, const float *b_scales,
    const float *bias, moeq_activation activation, const void *residual, void *z,
    const uint32_t *a_offsets, const int32_t *expert_ids, int64_t total_tokens, int64_t N,
    int64_t K, int32_t num_experts, int32_t max_tokens_per_expert, int32_t num_active_experts,
    moeq_stream_t stream) {
    (void)max_tokens_per_expert;
    if (!activation_ok(activation)) return MOEQ_ERR_INVALID_ARG;
    if (z && (z == c || z == residual)) return MOEQ_ERR_INVALID_ARG;
    moeq::GemmBlockArgs ga = {};
    ga.N = N;
    ga.K = K;
    ga.a = a;
    ga.b = b;
    ga.a_scales = a_scales;
    ga.b_scales = b_scales;
    ga.c = c;
    ga.bias = bias;
    ga.act = activation;
    ga.residual = residual;
    ga.z = z;
    return matmul_fp8_block_call(ga, a_offsets, expert_ids, total_tokens, num_experts,
                                 num_active_experts, stream);
}

static moeq_status epilogue_grad_sizes_ok(int64_t rows, int64_t N, int32_t groups) {
    if (rows < 0 || N <= 0 || N % 8 || groups < 0) return MOEQ_ERR_INVALID_ARG;
    if (rows >= (int64_t)1 << 31 || N >= (int64_t)1 << 31 || groups > moeq::kMaxGroups)
        return MOEQ_ERR_UNSUPPORTED;
    return MOEQ_OK;
}

int64_t moeq_grouped_epilogue_grad_workspace(int64_t total_tokens, int64_t N,
                                             int32_t num_active_experts) {
    if (epilogue_grad_sizes_ok(total_tokens, N, num_active_experts) != MOEQ_OK) return -1;
    return moeq::epilogue_grad_table_bytes(num_active_experts) +
           moeq::epilogue_grad_tiles(total_tokens, N, num_active_experts) * N * 4;
}

moeq_status moeq_grouped_epilogue_grad(const void *d_c, int64_t d_c_stride, const void *z,
                                       moeq_activation activation, uint8_t *q, float *scales,
                                       void *d_z, float *d_bias, const uint32_t *a_offsets,
                                       const int32_t *expert_ids, int64_t total_tokens, int64_t N,
                                       int32_t num_experts, int32_t num_active_experts,
                                       void *workspace, moeq_stream_t stream) {
    if (!groups_ok(a_offsets, expert_ids, num_experts, num_active_experts) ||
        !activation_ok(activation))
        return MOEQ_ERR_INVALID_ARG;
    const moeq_status st = epilogue_grad_sizes_ok(total_tokens, N, num_active_experts);
    if (st != MOEQ_OK) return st;
    if (num_experts > 65535) return MOEQ_ERR_UNSUPPORTED;
    if (!aligned16(d_bias) || !aligned16(workspace) || (d_bias && !workspace))
        return MOEQ_ERR_INVALID_ARG;
    const bool work = total_tokens > 0 && num_active_experts > 0;
    if (work && (!d_c || !aligned16(d_c) || d_c_stride < N || d_c_stride % 8 || !aligned16(z) ||
                 !z != (activation == MOEQ_ACT_NONE) || !aligned16(q) || !aligned16(scales) ||
                 !q != !scales || (q && N % 16) || !aligned16(d_z) || (!q && !d_z && !d_bias)))
        return MOEQ_ERR_INVALID_ARG;
    if (!work && !d_bias) return MOEQ_OK;
    uint32_t *err = device_error_ptr();
    if (!err) return cuda_status(cudaErrorInvalidDevice);
    moeq::EpilogueGradArgs g = {};
    g.groups = make_groups(a_offsets, nullptr, expert_ids, num_active_experts, num_experts,
                           total_tokens, 0);
    g.N = N;
    g.dc = d_c;
    g.z = z;
    g.dc_stride = d_c_stride;
    g.act = activation;
    g.q = q;
    g.scales = scales;
    g.dz = d_z;
    g.d_bias = d_bias;
    g.workspace = workspace;
    g.err = err;
    return cuda_status(moeq::launch_epilogue_grad(g, stream));
}

}  // extern "C"
