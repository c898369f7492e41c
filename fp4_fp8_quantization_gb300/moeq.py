"""Python binding of the moeq C ABI (``include/moeq.h``).

Argument marshalling only: each function checks that the tensors it is given
are CUDA tensors of the documented dtype and layout, passes their device
pointers and sizes to the function of the same name in ``libmoeq.so`` on the
current CUDA stream (or ``stream``), and raises ``MoeqError`` on a non-OK
status.  Every step of the computation runs in the library's CUDA kernels;
there is no other implementation, and importing a function whose library is
missing raises.
"""
import ctypes
import os

import torch

# The in-tree library, or another build of it named by MOEQ_LIB (e.g. one
# compiled with different tile options by build.build(variant_dir, flags)).
_LIB_PATH = os.environ.get("MOEQ_LIB") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libmoeq.so")
_lib = None

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # moeq_dtype
SCORES = {"softmax": 0, "sigmoid": 1}                              # moeq_score
GROUP_SCORES = {"max": 0, "top2": 1}                               # moeq_group_score
ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}   # moeq_activation
FORMATS = {"nvfp4": 0, "mxfp4": 1, "mxfp8": 2}
STATUS = {0: "MOEQ_OK", 1: "MOEQ_ERR_INVALID_ARG", 2: "MOEQ_ERR_UNSUPPORTED",
          3: "MOEQ_ERR_CUDA", 4: "MOEQ_ERR_DEVICE"}
DEVERR_BAD_OFFSETS, DEVERR_BAD_EXPERT, DEVERR_SCALE_ROWS, DEVERR_TIMEOUT, DEVERR_BAD_INDEX = 1, 2, 4, 8, 16
DEVERR_BOUNDS = 32   # debug builds only: a store outside its buffer was skipped

_P, _I64, _I32, _U32P = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(ctypes.c_uint32)
_F = ctypes.c_float
_SIGNATURES = {
    "moeq_grouped_amax_scale": [_P, _I64, _I64, _I64, _P, _P, _P, _I32, _I32, _P],
    "moeq_grouped_quantize": [_I32, _P, _I64, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P,
                              _I32, _I32, _I32, _P],
    "moeq_grouped_amax_scale_gather": [_P, _I64, _I64, _I64, _P, _I32, _I64, _P, _P, _P, _I32,
                                       _I32, _P],
    "moeq_grouped_quantize_gather": [_I32, _P, _I64, _I64, _I64, _P, _I32, _I64, _P, _P, _I64,
                                     _P, _P, _P, _P, _I32, _I32, _I32, _P],
    "moeq_padded_scale_offsets": [_P, _P, _I32, _P],
    "moeq_grouped_matmul_rowwise_fp8": [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64,
                                        _I32, _I32, _I32, _P],
    "moeq_grouped_matmul_blockscaled": [_I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64,
                                        _I64, _I64, _I32, _I32, _I32, _P],
    "moeq_swiglu_quantize": [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32, _P],
    "moeq_swiglu_quantize_mx": [_I32, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32,
                                _P],
    "moeq_grouped_matmul_swiglu": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64,
                                   _I64, _I64, _I32, _I32, _I32, _P],
    "moeq_grouped_matmul_swiglu_mx": [_I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64,
                                      _I64, _I64, _I32, _I32, _I32, _P],
    "moeq_sf_swizzle": [_P, _P, _I64, _I64, _I64, _P],
    "moeq_sf_unswizzle": [_P, _P, _I64, _I64, _I64, _P],
    "moeq_interleave_gate_up": [_P, _P, _P, _I64, _I64, _I64, _P],
    "moeq_route_topk": [_P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _I32, _P],
    "moeq_quantize_topk": [_I32, _P, _I64, _I64, _I64, _P, _I32, _P, _P, _P, _P, _I32, _P, _P,
                           _I64, _P],
    "moeq_dispatch_scale_rows": [_I64, _I32, _I32, _I32],
    "moeq_grouped_amax_scale_topk": [_P, _I64, _I64, _I64, _P, _I32, _P, _I32, _P],
    "moeq_dispatch_mxfp4": [_P, _I64, _I64, _I64, _P, _I32, _I32, _P, _P, _I64, _P, _P, _P, _P,
                            _P, _I32, _P],
    "moeq_gate_topk": [_I32, _P, _I64, _I64, _I32, _I32, _I32, _F, _P, _P, _P],
    "moeq_gate_topk_grad": [_I32, _P, _I64, _I64, _I32, _I32, _I32, _F, _P, _P, _P, _P],
    "moeq_gate_group_topk": [_I32, _P, _I64, _I64, _I32, _P, _I32, _I32, _I32, _I32, _I32, _I32,
                             _F, _P, _P, _P],
    "moeq_gate_group_topk_grad": [_I32, _P, _I64, _I64, _I32, _I32, _I32, _I32, _F, _P, _P, _P,
                                  _P],
    "moeq_permute_topk": [_I32, _P, _I64, _I64, _I64, _P, _I32, _P, _P, _I64, _P],
    "moeq_permute_topk_grad": [_I32, _P, _I64, _I64, _I64, _P, _I32, _P, _P, _P, _I64, _P, _P],
    "moeq_combine_topk": [_I32, _P, _I64, _I64, _I64, _P, _I32, _P, _P, _P],
    "moeq_combine_topk_grad": [_I32, _P, _I64, _I64, _I64, _P, _I32, _P, _P, _I64, _P, _P, _P],
    "moeq_quantize_fp8_block": [_P, _I64, _I64, _I64, _P, _P, _P],
    "moeq_quantize_fp8_block_topk": [_P, _I64, _I64, _I64, _P, _I32, _P, _P, _I64, _P],
    "moeq_swiglu_quantize_fp8_block": [_P, _I64, _I64, _P, _P, _P],
    "moeq_quantize_fp8_block_weight": [_P, _I64, _I64, _I64, _P, _P, _P],
    "moeq_add_rms_norm": [_I32, _P, _I64, _P, _I64, _I64, _I64, _P, _F, _P, _P, _P, _P, _I32, _P,
                          _P],
    "moeq_add_rms_norm_grad_workspace": [_I64, _I64],
    "moeq_add_rms_norm_grad": [_I32, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P,
                               _P],
    "moeq_grouped_matmul_fp8_block": [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32,
                                      _I32, _P],
    "moeq_grouped_matmul_fp8_block_epilogue": [_P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _I64,
                                               _I64, _I64, _I32, _I32, _I32, _P],
    "moeq_grouped_epilogue_grad": [_P, _I64, _P, _I32, _P, _P, _P, _P, _P, _P, _I64, _I64, _I32,
                                   _I32, _P, _P],
    "moeq_grouped_epilogue_grad_workspace": [_I64, _I64, _I32],
    "moeq_get_device_error": [_P, _U32P],
    "moeq_clear_device_error": [_P],
    "moeq_last_cuda_error": [],
    "moeq_status_string": [ctypes.c_int],
}
EXPORTS = tuple(_SIGNATURES)


class MoeqError(RuntimeError):
    def __init__(self, fn, status):
        code = lib().moeq_last_cuda_error() if status == 3 else 0
        super().__init__(f"{fn}: {STATUS.get(status, status)}" + (f" (cuda error {code})" if code else ""))
        self.status = status


def lib():
    """The loaded libmoeq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "python -m fp4_fp8_quantization_gb300.build")
        L = ctypes.CDLL(_LIB_PATH)
        for name, args in _SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.moeq_status_string.restype = ctypes.c_char_p
        L.moeq_dispatch_scale_rows.restype = ctypes.c_int64
        L.moeq_add_rms_norm_grad_workspace.restype = ctypes.c_int64
        L.moeq_grouped_epilogue_grad_workspace.restype = ctypes.c_int64
        _lib = L
    return _lib


# The handle of the current stream without building a torch.cuda.Stream
# (0.2 us a call against 2.9).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _raw_device is not None:
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _ptr_rows(t, dtype, name):
    """Pointer of a 2-D tensor whose rows may be strided (unit element
    stride, row stride >= row length)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: must be 2-D with unit column stride")
    return t.data_ptr()


def _call(fn, *args):
    st = getattr(_lib or lib(), fn)(*args)
    if st != 0:
        raise MoeqError(fn, st)


def _fmt(fmt):
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


_U8 = (torch.uint8, torch.float8_e4m3fn)
_U32 = (torch.uint32, torch.int32)


def grouped_amax_scale(inp, row_offsets, expert_ids, tensor_scale_out, num_experts,
                       num_active_experts=None, stream=None):
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    _call("moeq_grouped_amax_scale", _ptr_rows(inp, torch.bfloat16, "inp"), inp.stride(0),
          inp.shape[0], inp.shape[1], _ptr(row_offsets, _U32), _ptr(expert_ids, torch.int32),
          _ptr(tensor_scale_out, torch.float32), num_experts, G, _stream(stream))


def grouped_quantize(fmt, inp, out, scales, row_offsets, scales_offsets, expert_ids,
                     tensor_scale, num_experts, scale_rows_total, max_tokens_per_expert=0,
                     num_active_experts=None, stream=None):
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    _call("moeq_grouped_quantize", _fmt(fmt), _ptr_rows(inp, torch.bfloat16, "inp"), inp.stride(0),
          inp.shape[0], inp.shape[1], _ptr(out, _U8, "out"), _ptr(scales, _U8, "scales"),
          scale_rows_total, _ptr(row_offsets, _U32), _ptr(scales_offsets, _U32),
          _ptr(expert_ids, torch.int32), _ptr(tensor_scale, torch.float32), num_experts,
          max_tokens_per_expert, G, _stream(stream))


def grouped_amax_scale_gather(inp, indices, indices_divisor, row_offsets, expert_ids,
                              tensor_scale_out, num_experts, num_active_experts=None,
                              stream=None):
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    _call("moeq_grouped_amax_scale_gather", _ptr_rows(inp, torch.bfloat16, "inp"), inp.stride(0),
          inp.shape[0], inp.shape[1], _ptr(indices, torch.int32, "indices"), indices_divisor,
          indices.numel(), _ptr(row_offsets, _U32), _ptr(expert_ids, torch.int32),
          _ptr(tensor_scale_out, torch.float32), num_experts, G, _stream(stream))


def grouped_quantize_gather(fmt, inp, indices, indices_divisor, out, scales, row_offsets,
                            scales_offsets, expert_ids, tensor_scale, num_experts,
                            scale_rows_total, max_tokens_per_expert=0, num_active_experts=None,
                            stream=None):
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    _call("moeq_grouped_quantize_gather", _fmt(fmt), _ptr_rows(inp, torch.bfloat16, "inp"),
          inp.stride(0), inp.shape[0], inp.shape[1], _ptr(indices, torch.int32, "indices"),
          indices_divisor, indices.numel(), _ptr(out, _U8, "out"), _ptr(scales, _U8, "scales"),
          scale_rows_total, _ptr(row_offsets, _U32), _ptr(scales_offsets, _U32),
          _ptr(expert_ids, torch.int32), _ptr(tensor_scale, torch.float32), num_experts,
          max_tokens_per_expert, G, _stream(stream))


def padded_scale_offsets(row_offsets, scales_offsets, num_active_experts=None, stream=None):
    G = row_offsets.numel() - 1 if num_active_experts is None else num_active_experts
    _call("moeq_padded_scale_offsets", _ptr(row_offsets, _U32), _ptr(scales_offsets, _U32), G,
          _stream(stream))


def sf_swizzle(tiled, logical, stream=None):
    """logical uint8 [rows, kv] or [batch, rows, kv] -> the tiled block-scale
    layout in `tiled` (uint8, batch * sf_bytes(rows, kv) bytes)."""
    batch, rows, kv = (1, *logical.shape) if logical.dim() == 2 else logical.shape
    if tiled.numel() != batch * sf_bytes(rows, kv):
        raise ValueError("tiled: expected batch * sf_bytes(rows, kv) bytes")
    _call("moeq_sf_swizzle", _ptr(tiled, _U8, "tiled"), _ptr(logical, _U8, "logical"), batch,
          rows, kv, _stream(stream))


def sf_unswizzle(logical, tiled, stream=None):
    """The inverse of sf_swizzle: fills logical uint8 [rows, kv] or
    [batch, rows, kv] from the tiled buffer."""
    batch, rows, kv = (1, *logical.shape) if logical.dim() == 2 else logical.shape
    if tiled.numel() != batch * sf_bytes(rows, kv):
        raise ValueError("tiled: expected batch * sf_bytes(rows, kv) bytes")
    _call("moeq_sf_unswizzle", _ptr(logical, _U8, "logical"), _ptr(tiled, _U8, "tiled"), batch,
          rows, kv, _stream(stream))


def interleave_gate_up(out, gate, up, stream=None):
    """out[b, 2j] = gate[b, j], out[b, 2j + 1] = up[b, j]: uint8 gate, up
    [batch, rows, row_bytes] (or 2-D), out [batch, 2 * rows, row_bytes]."""
    if gate.shape != up.shape:
        raise ValueError("gate and up must have the same shape")
    batch, rows, rb = (1, *gate.shape) if gate.dim() == 2 else gate.shape
    if out.numel() != batch * 2 * rows * rb:
        raise ValueError("out: expected batch * 2 * rows * row_bytes bytes")
    _call("moeq_interleave_gate_up", _ptr(out, _U8, "out"), _ptr(gate, _U8, "gate"),
          _ptr(up, _U8, "up"), batch, rows, rb, _stream(stream))


def route_topk(topk_ids, row_offsets, expert_ids, src_info, scales_offsets=None, slot_rows=0,
               stream=None, dst_info=None):
    """Routes the choices of topk_ids (int32 [num_tokens, top_k]) to the
    groups of their experts: row_offsets (int32/uint32 [E + 1]), expert_ids
    (int32 [E]), src_info (int32 [num_tokens * top_k]) and, if given,
    scales_offsets ([E + 1]: padded, or slots of slot_rows rows) and
    dst_info (int32 [num_tokens * top_k], the row of each choice)."""
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids: expected [num_tokens, top_k]")
    E = expert_ids.numel()
    if row_offsets.numel() != E + 1 or src_info.numel() < topk_ids.numel():
        raise ValueError("row_offsets [E + 1] and src_info [num_tokens * top_k] expected")
    _call("moeq_route_topk", _ptr(topk_ids, torch.int32, "topk_ids"), topk_ids.shape[0],
          topk_ids.shape[1], E, _ptr(row_offsets, _U32, "row_offsets"),
          _ptr(expert_ids, torch.int32, "expert_ids"), _ptr(src_info, torch.int32, "src_info"),
          _ptr(dst_info, torch.int32, "dst_info"), _ptr(scales_offsets, _U32, "scales_offsets"),
          slot_rows, _stream(stream))


def grouped_amax_scale_topk(tokens, topk_ids, tensor_scale_out, num_experts, stream=None):
    """Per-expert NVFP4 tensor scales from bf16 tokens [num_tokens, K] and
    their top-k expert ids (int32 [num_tokens, top_k]); each token read once."""
    if topk_ids.dim() != 2 or topk_ids.shape[0] != tokens.shape[0]:
        raise ValueError("topk_ids: expected [num_tokens, top_k]")
    _call("moeq_grouped_amax_scale_topk", _ptr_rows(tokens, torch.bfloat16, "tokens"),
          tokens.stride(0), tokens.shape[0], tokens.shape[1],
          _ptr(topk_ids, torch.int32, "topk_ids"), topk_ids.shape[1],
          _ptr(tensor_scale_out, torch.float32, "tensor_scale_out"), num_experts,
          _stream(stream))


def dispatch_scale_rows(num_tokens, top_k, num_experts, slot_rows=0):
    """Logical scale rows dispatch_mxfp4 needs for these sizes."""
    n = lib().moeq_dispatch_scale_rows(num_tokens, top_k, num_experts, slot_rows)
    if n < 0:
        raise ValueError("invalid sizes")
    return n


def quantize_topk(fmt, tokens, topk_ids, dst_info, out, scales, row_offsets, scales_offsets,
                  tensor_scale, num_experts, stream=None):
    """Token-major quantization of routed tokens (the bytes of
    grouped_quantize_gather on the routed rows, each token read once):
    tokens bf16 [num_tokens, K]; topk_ids int32 [num_tokens, top_k];
    dst_info, row_offsets, scales_offsets from route_topk; out
    [num_tokens * top_k, K / 2] (FP4) or [.., K] (MXFP8)."""
    if topk_ids.dim() != 2 or topk_ids.shape[0] != tokens.shape[0]:
        raise ValueError("topk_ids: expected [num_tokens, top_k]")
    T, K = tokens.shape
    v = 16 if fmt == "nvfp4" else 32
    rows = scales.numel() // max(1, sf_bytes(128, K // v)) * 128
    _call("moeq_quantize_topk", _fmt(fmt), _ptr_rows(tokens, torch.bfloat16, "tokens"),
          tokens.stride(0), T, K, _ptr(topk_ids, torch.int32, "topk_ids"), topk_ids.shape[1],
          _ptr(dst_info, torch.int32, "dst_info"), _ptr(row_offsets, _U32, "row_offsets"),
          _ptr(scales_offsets, _U32, "scales_offsets"),
          _ptr(tensor_scale, torch.float32, "tensor_scale"), num_experts,
          _ptr(out, _U8, "out"), _ptr(scales, _U8, "scales"), rows, _stream(stream))


def dispatch_mxfp4(tokens, topk_ids, out, scales, row_offsets, expert_ids, src_info,
                   scales_offsets, slot_rows=0, stream=None, dst_info=None):
    """Single-rank expert dispatch: route_topk, then MXFP4 quantization of
    the routed rows (row r is token src_info[r] // top_k).  tokens bf16
    [num_tokens, hidden]; out uint8 [num_tokens * top_k, hidden / 2]; scales
    the tiled E8M0 buffer (sf_bytes(rows, hidden / 32) bytes for
    rows = dispatch_scale_rows(...) or more, a multiple of 128)."""
    if topk_ids.dim() != 2 or topk_ids.shape[0] != tokens.shape[0]:
        raise ValueError("topk_ids: expected [num_tokens, top_k]")
    T, H = tokens.shape
    E = expert_ids.numel()
    if out.numel() < topk_ids.numel() * (H // 2) or row_offsets.numel() != E + 1:
        raise ValueError("out [num_tokens * top_k, hidden / 2] and row_offsets [E + 1] expected")
    rows = scales.numel() // max(1, sf_bytes(128, H // 32)) * 128
    if dst_info is None:   # the inverse routing map, device memory owned by the caller
        dst_info = torch.empty(topk_ids.numel(), dtype=torch.int32, device=tokens.device)
    _call("moeq_dispatch_mxfp4", _ptr_rows(tokens, torch.bfloat16, "tokens"), tokens.stride(0),
          T, H, _ptr(topk_ids, torch.int32, "topk_ids"), topk_ids.shape[1], E,
          _ptr(out, _U8, "out"), _ptr(scales, _U8, "scales"), rows,
          _ptr(row_offsets, _U32, "row_offsets"), _ptr(expert_ids, torch.int32, "expert_ids"),
          _ptr(src_info, torch.int32, "src_info"), _ptr(dst_info, torch.int32, "dst_info"),
          _ptr(scales_offsets, _U32, "scales_offsets"), slot_rows, _stream(stream))


def grouped_matmul_rowwise_fp8(c, a, b, a_scales, b_scales, a_offsets, expert_ids,
                               max_tokens_per_expert=0, num_active_experts=None, stream=None):
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    E, N, K = b.shape
    _call("moeq_grouped_matmul_rowwise_fp8", _ptr(c, torch.bfloat16, "c"), _ptr(a, _U8, "a"),
          _ptr(b, _U8, "b"), _ptr(a_scales, torch.float32), _ptr(b_scales, torch.float32),
          _ptr(a_offsets, _U32), _ptr(expert_ids, torch.int32), a.shape[0], N, K, E,
          max_tokens_per_expert, G, _stream(stream))


def grouped_matmul_blockscaled(fmt, c, a, a_sf, b, b_sf, expert_scales, a_offsets,
                               a_scales_offsets, expert_ids, N, K, scale_rows_total,
                               max_tokens_per_expert=0, num_active_experts=None, stream=None):
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    _call("moeq_grouped_matmul_blockscaled", _fmt(fmt), _ptr(c, torch.bfloat16, "c"),
          _ptr(a, _U8, "a"), _ptr(a_sf, _U8, "a_sf"), _ptr(b, _U8, "b"), _ptr(b_sf, _U8, "b_sf"),
          _ptr(expert_scales, torch.float32), _ptr(a_offsets, _U32), _ptr(a_scales_offsets, _U32),
          _ptr(expert_ids, torch.int32), a.shape[0], scale_rows_total, N, K, b.shape[0],
          max_tokens_per_expert, G, _stream(stream))


def swiglu_quantize(c_packed, c_sf, y, out_tensor_scale, a_offsets, a_scales_offsets,
                    expert_ids, num_experts, scale_rows_total, max_tokens_per_expert=0,
                    num_active_experts=None, stream=None):
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    _call("moeq_swiglu_quantize", _ptr(c_packed, _U8), _ptr(c_sf, _U8),
          _ptr(y, torch.bfloat16, "y"), _ptr(out_tensor_scale, torch.float32),
          _ptr(a_offsets, _U32), _ptr(a_scales_offsets, _U32), _ptr(expert_ids, torch.int32),
          y.shape[0], scale_rows_total, y.shape[1] // 2, num_experts, max_tokens_per_expert, G,
          _stream(stream))


def swiglu_quantize_mx(fmt, c_q, c_sf, y, a_offsets, a_scales_offsets, expert_ids, num_experts,
                       scale_rows_total, max_tokens_per_expert=0, num_active_experts=None,
                       stream=None):
    """Chained SwiGLU + MXFP4 / MXFP8 requantization (fmt "mxfp4" / "mxfp8")."""
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    _call("moeq_swiglu_quantize_mx", _fmt(fmt), _ptr(c_q, _U8), _ptr(c_sf, _U8),
          _ptr(y, torch.bfloat16, "y"), _ptr(a_offsets, _U32), _ptr(a_scales_offsets, _U32),
          _ptr(expert_ids, torch.int32), y.shape[0], scale_rows_total, y.shape[1] // 2,
          num_experts, max_tokens_per_expert, G, _stream(stream))


def grouped_matmul_swiglu(c_packed, c_sf, a, a_sf, b, b_sf, expert_scales, out_tensor_scale,
                          a_offsets, a_scales_offsets, expert_ids, I, K, scale_rows_total,
                          max_tokens_per_expert=0, num_active_experts=None, stream=None,
                          a_row_scales=None):
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    _call("moeq_grouped_matmul_swiglu", _ptr(c_packed, _U8), _ptr(c_sf, _U8), _ptr(a, _U8),
          _ptr(a_sf, _U8), _ptr(b, _U8), _ptr(b_sf, _U8), _ptr(expert_scales, torch.float32),
          _ptr(out_tensor_scale, torch.float32),
          _ptr(a_row_scales, torch.bfloat16, "a_row_scales"), _ptr(a_offsets, _U32),
          _ptr(a_scales_offsets, _U32), _ptr(expert_ids, torch.int32), a.shape[0],
          scale_rows_total, I, K, b.shape[0], max_tokens_per_expert, G, _stream(stream))


def grouped_matmul_swiglu_mx(fmt, c_q, c_sf, a, a_sf, b, b_sf, expert_scales, a_offsets,
                             a_scales_offsets, expert_ids, I, K, scale_rows_total,
                             max_tokens_per_expert=0, num_active_experts=None, stream=None):
    """Fused grouped MX matmul + SwiGLU + MX requantization (fmt "mxfp4" / "mxfp8")."""
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    _call("moeq_grouped_matmul_swiglu_mx", _fmt(fmt), _ptr(c_q, _U8), _ptr(c_sf, _U8),
          _ptr(a, _U8), _ptr(a_sf, _U8), _ptr(b, _U8), _ptr(b_sf, _U8),
          _ptr(expert_scales, torch.float32), _ptr(a_offsets, _U32),
          _ptr(a_scales_offsets, _U32), _ptr(expert_ids, torch.int32), a.shape[0],
          scale_rows_total, I, K, b.shape[0], max_tokens_per_expert, G, _stream(stream))


def _rows_of(t, name, shape=None, dtype=None):
    """Pointer of a 2-D CUDA tensor with unit column stride (rows may be
    strided) of one of DTYPES, or of dtype, and of the given shape."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2
            and (t.dtype in DTYPES if dtype is None else t.dtype is dtype)
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype not in DTYPES if dtype is None else t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype or tuple(DTYPES)}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape or '2-D'}")
    n, m = t.shape
    if m > 1 and t.stride(1) != 1 or n > 1 and t.stride(0) < m:
        raise ValueError(f"{name}: must have unit column stride")
    return t.data_ptr()


def _row_stride(t):
    # a single row has no stride to speak of
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _shaped(t, shape, dtype, name, optional=False):
    """Pointer of a contiguous CUDA tensor of this shape and dtype; None is
    None where that is allowed."""
    # the checks in one expression: a call has many arguments and a small one
    # takes little more than their checks
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.shape == shape
            and (t.dtype is dtype or (type(dtype) is tuple and t.dtype in dtype))
            and t.is_contiguous()):
        return t.data_ptr()
    if t is None and optional:
        return None
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: required" if t is None else f"{name}: expected a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return _ptr(t, dtype, name)


def _dtype_code(t, name):
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {tuple(DTYPES)}")
    return code


def _choices(dst_info, num_tokens):
    if dst_info.dim() != 2 or dst_info.shape[0] != num_tokens or dst_info.shape[1] < 1:
        raise ValueError("dst_info: expected [num_tokens, top_k]")
    return dst_info.shape[1]


def gate_topk(logits, topk_ids, weights, normalize=True, scale=1.0, stream=None):
    """The router: topk_ids (int32 [num_tokens, top_k], out) are the largest
    logits of each token (ties to the lowest index) and weights (fp32, out)
    their softmax weights times scale, over the chosen (normalize) or over all
    experts.  logits bf16 / fp16 / fp32 [num_tokens, num_experts], -inf for a
    masked expert; a token with too few others gets id -1 and weight 0."""
    p = _rows_of(logits, "logits")
    T, E = logits.shape
    k = _choices(topk_ids, T)
    _call("moeq_gate_topk", DTYPES[logits.dtype], p, _row_stride(logits), T, E, k, bool(normalize),
          scale, _ptr(topk_ids, torch.int32, "topk_ids"),
          _shaped(weights, (T, k), torch.float32, "weights"), _stream(stream))


def gate_topk_grad(logits, topk_ids, d_weights, d_logits, normalize=True, scale=1.0, stream=None):
    """Gradient of gate_topk's weights: d_logits (out, the logits' dtype,
    contiguous) from d_weights fp32 [num_tokens, top_k] and the logits and
    topk_ids of the forward call."""
    p = _rows_of(logits, "logits")
    T, E = logits.shape
    k = _choices(topk_ids, T)
    _call("moeq_gate_topk_grad", DTYPES[logits.dtype], p, _row_stride(logits), T, E, k,
          bool(normalize), scale, _ptr(topk_ids, torch.int32, "topk_ids"),
          _shaped(d_weights, (T, k), torch.float32, "d_weights"),
          _shaped(d_logits, (T, E), logits.dtype, "d_logits"), _stream(stream))


def _one_of(names, name, what):
    code = names.get(name)
    if code is None:
        raise ValueError(f"{what}: {name!r}, expected one of {tuple(names)}")
    return code


# The checks of the calls below: they launch on the current device, where every
# tensor lives.  A small call takes little more than its checks, so that what is
# right is seen in one expression (a host tensor's device is -1) and what is
# wrong is looked at again for its message.

def _on_current_device(dev):
    if dev != (_raw_device() if _raw_device is not None else torch.cuda.current_device()):
        raise ValueError(f"tensors on cuda:{dev}: expected the current device")


def _matrix(t, name, dtype=None, shape=None, dev=None):
    """(pointer, row stride, device) of a 2-D CUDA tensor, as _rows_of."""
    try:
        if ((t.dtype in DTYPES if dtype is None else t.dtype is dtype) and t.is_contiguous()
                and (t.dim() == 2 if shape is None else t.shape == shape)):
            at = t.get_device()
            if at >= 0 and (dev is None or at == dev):
                return t.data_ptr(), t.shape[1], at
    except AttributeError:
        pass
    p = _rows_of(t, name, shape, dtype)
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")
    return p, _row_stride(t), t.get_device()


def _array(t, shape, dtype, dev, name):
    """Pointer of a contiguous tensor of this shape and dtype on device dev."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _shaped(t, shape, dtype, name)
    raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")


def _array_of(t, shape, dtypes, dev, name):
    """_array of one of two dtypes."""
    return _array(t, shape, dtypes[1 if t.dtype is dtypes[1] else 0], dev, name)


def _groups(a_offsets, expert_ids, num_active_experts, dev):
    """(pointer, pointer, groups) of a ragged group description."""
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    if expert_ids.numel() < G or a_offsets.numel() < G + 1:
        raise ValueError(f"a_offsets, expert_ids: too short for {G} groups")
    return (_array_of(a_offsets, a_offsets.shape, _U32, dev, "a_offsets"),
            _array(expert_ids, expert_ids.shape, torch.int32, dev, "expert_ids"), G)


def _checked(fn, status):
    if status != 0:
        raise MoeqError(fn, status)


def gate_group_topk(logits, topk_ids, weights, bias=None, score="sigmoid", num_groups=1,
                    topk_groups=None, group_score="top2", normalize=True, scale=1.0, stream=None):
    """The router with scores ("sigmoid" or "softmax" of the logits), a balance
    bias (fp32 [num_experts] or None: added to the scores for the choice, not in
    the weights) and groups: of num_groups groups of consecutive experts the
    topk_groups (None: all) of the largest value are kept, the value being the
    best score with bias ("max") or the sum of the best two ("top2").  topk_ids
    (int32 [num_tokens, top_k], out) are the best experts of those, the best
    first, ties to the lowest index; weights (fp32, out) their scores, divided by
    their sum (normalize), times scale.  logits bf16 / fp16 / fp32 [num_tokens,
    num_experts], -inf for a masked expert; id -1 and weight 0 where none is left."""
    p, stride, dev = _matrix(logits, "logits")
    T, E = logits.shape
    k = _choices(topk_ids, T)
    shape = (T, k)
    ids = _array(topk_ids, shape, torch.int32, dev, "topk_ids")
    w = _array(weights, shape, torch.float32, dev, "weights")
    b = None if bias is None else _array(bias, (E,), torch.float32, dev, "bias")
    _on_current_device(dev)
    _checked("moeq_gate_group_topk", (_lib or lib()).moeq_gate_group_topk(
        DTYPES[logits.dtype], p, stride, T, E, b, _one_of(SCORES, score, "score"), num_groups,
        num_groups if topk_groups is None else topk_groups,
        _one_of(GROUP_SCORES, group_score, "group_score"), k, bool(normalize), scale, ids, w,
        _stream(stream)))


def gate_group_topk_grad(logits, topk_ids, d_weights, d_logits, score="sigmoid", normalize=True,
                         scale=1.0, stream=None):
    """Gradient of gate_group_topk's weights, the choice taken as fixed: d_logits
    (out, the logits' dtype, contiguous, not over the logits) from d_weights fp32
    [num_tokens, top_k] and the logits and topk_ids of the forward call."""
    p, stride, dev = _matrix(logits, "logits")
    T, E = logits.shape
    k = _choices(topk_ids, T)
    shape = (T, k)
    ids = _array(topk_ids, shape, torch.int32, dev, "topk_ids")
    dw = _array(d_weights, shape, torch.float32, dev, "d_weights")
    dx = _array(d_logits, (T, E), logits.dtype, dev, "d_logits")
    _on_current_device(dev)
    _checked("moeq_gate_group_topk_grad", (_lib or lib()).moeq_gate_group_topk_grad(
        DTYPES[logits.dtype], p, stride, T, E, _one_of(SCORES, score, "score"), k, bool(normalize),
        scale, ids, dw, dx, _stream(stream)))


def permute_topk(tokens, dst_info, rows, weights=None, stream=None):
    """Tokens to their experts' rows: rows[dst_info[t, j]] = weights[t, j] *
    tokens[t] (weights fp32 [num_tokens, top_k], or None: copies).  tokens
    bf16 / fp16 / fp32 [num_tokens, hidden]; dst_info int32 [num_tokens,
    top_k] from route_topk; rows (out) of the tokens' dtype [rows, hidden]."""
    p = _rows_of(tokens, "tokens")
    T, H = tokens.shape
    k = _choices(dst_info, T)
    _call("moeq_permute_topk", DTYPES[tokens.dtype], p, _row_stride(tokens), T, H,
          _ptr(dst_info, torch.int32, "dst_info"), k,
          _shaped(weights, (T, k), torch.float32, "weights", True),
          _shaped(rows, (rows.shape[0], H), tokens.dtype, "rows"), rows.shape[0],
          _stream(stream))


def permute_topk_grad(d_rows, dst_info, d_tokens, weights=None, tokens=None, d_weights=None,
                      stream=None):
    """Gradient of permute_topk: d_tokens[t] (out) = the sum over j of
    weights[t, j] * d_rows[dst_info[t, j]]; with d_weights (out, fp32
    [num_tokens, top_k]) also <tokens[t], d_rows[dst_info[t, j]]>."""
    T, H = d_tokens.shape
    k = _choices(dst_info, T)
    if d_weights is not None and tokens is None:
        raise ValueError("tokens: required for d_weights")
    _call("moeq_permute_topk_grad", _dtype_code(d_tokens, "d_tokens"),
          _shaped(d_rows, (d_rows.shape[0], H), d_tokens.dtype, "d_rows"), d_rows.shape[0], T, H,
          _ptr(dst_info, torch.int32, "dst_info"), k,
          _shaped(weights, (T, k), torch.float32, "weights", True),
          _shaped(d_tokens, (T, H), d_tokens.dtype, "d_tokens"),
          None if tokens is None else _rows_of(tokens, "tokens", (T, H), d_tokens.dtype),
          H if tokens is None else _row_stride(tokens),
          _shaped(d_weights, (T, k), torch.float32, "d_weights", True), _stream(stream))


def combine_topk(rows, dst_info, out, weights=None, stream=None):
    """Rows back to their tokens: out[t] = the sum over j of weights[t, j] *
    rows[dst_info[t, j]] (weights None: 1).  rows bf16 / fp16 / fp32 [rows,
    hidden]; out of the same dtype [num_tokens, hidden]."""
    T, H = out.shape
    k = _choices(dst_info, T)
    _call("moeq_combine_topk", _dtype_code(out, "out"),
          _shaped(rows, (rows.shape[0], H), out.dtype, "rows"), rows.shape[0], T, H,
          _ptr(dst_info, torch.int32, "dst_info"), k,
          _shaped(weights, (T, k), torch.float32, "weights", True),
          _shaped(out, (T, H), out.dtype, "out"), _stream(stream))


def combine_topk_grad(d_out, dst_info, d_rows, weights=None, rows=None, d_weights=None,
                      stream=None):
    """Gradient of combine_topk: d_rows[dst_info[t, j]] (out) = weights[t, j]
    * d_out[t]; with d_weights (out, fp32 [num_tokens, top_k]) also
    <d_out[t], rows[dst_info[t, j]]>."""
    p = _rows_of(d_out, "d_out")
    T, H = d_out.shape
    k = _choices(dst_info, T)
    if d_weights is not None and rows is None:
        raise ValueError("rows: required for d_weights")
    n = d_rows.shape[0]
    _call("moeq_combine_topk_grad", DTYPES[d_out.dtype], p, _row_stride(d_out), T, H,
          _ptr(dst_info, torch.int32, "dst_info"), k,
          _shaped(weights, (T, k), torch.float32, "weights", True),
          _shaped(d_rows, (n, H), d_out.dtype, "d_rows"), n,
          _shaped(rows, (n, H), d_out.dtype, "rows", True),
          _shaped(d_weights, (T, k), torch.float32, "d_weights", True), _stream(stream))


def _blocks128(n):
    return (n + 127) // 128


def quantize_fp8_block(inp, out, scales, stream=None):
    """E4M3 with one fp32 scale per 128 elements of a row: inp bf16 [rows, K]
    -> out (uint8 / float8_e4m3fn [rows, K]), scales fp32 [rows, ceil(K / 128)]."""
    p = _rows_of(inp, "inp", dtype=torch.bfloat16)
    T, K = inp.shape
    _call("moeq_quantize_fp8_block", p, _row_stride(inp), T, K,
          _shaped(out, (T, K), _U8, "out"),
          _shaped(scales, (T, _blocks128(K)), torch.float32, "scales"),
          _stream(stream))


def quantize_fp8_block_topk(tokens, dst_info, out, scales, stream=None):
    """quantize_fp8_block of routed tokens: rows dst_info[t, j] of out and
    scales are token t's, each token read and quantized once."""
    p = _rows_of(tokens, "tokens", dtype=torch.bfloat16)
    T, K = tokens.shape
    k = _choices(dst_info, T)
    n = out.shape[0]
    _call("moeq_quantize_fp8_block_topk", p, _row_stride(tokens), T, K,
          _ptr(dst_info, torch.int32, "dst_info"), k, _shaped(out, (n, K), _U8, "out"),
          _shaped(scales, (n, _blocks128(K)), torch.float32, "scales"), n,
          _stream(stream))


def swiglu_quantize_fp8_block(y, out, scales, stream=None):
    """quantize_fp8_block of silu(gate) * up: y bf16 [rows, 2 I] with column
    2j = gate_j, 2j + 1 = up_j; out [rows, I], scales [rows, ceil(I / 128)]."""
    T, I = y.shape[0], y.shape[1] // 2
    _call("moeq_swiglu_quantize_fp8_block", _shaped(y, (T, 2 * I), torch.bfloat16, "y"), T, I,
          _shaped(out, (T, I), _U8, "out"),
          _shaped(scales, (T, _blocks128(I)), torch.float32, "scales"),
          _stream(stream))


def quantize_fp8_block_weight(w, out, scales, stream=None):
    """Weights in E4M3 with one fp32 scale per 128 x 128 block: w bf16 [E, N,
    K] -> out of that shape, scales fp32 [E, ceil(N / 128), ceil(K / 128)]."""
    E, N, K = w.shape
    _call("moeq_quantize_fp8_block_weight", _ptr(w, torch.bfloat16, "w"), E, N, K,
          _shaped(out, (E, N, K), _U8, "out"),
          _shaped(scales, (E, _blocks128(N), _blocks128(K)), torch.float32,
                  "scales"), _stream(stream))


def _workspace(workspace, need, stream, like, dev):
    """(pointer, tensor) of a workspace of at least `need` bytes: the caller's, or
    a new one (freed in the current stream's order by PyTorch's allocator, so not
    for another stream)."""
    if need < 0:
        raise ValueError("sizes that the call does not take")
    if workspace is None:
        if stream is not None:
            raise ValueError("workspace: required with a stream")
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
        return workspace.data_ptr(), workspace
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace: {need} bytes expected")
    return _array(workspace, workspace.shape, workspace.dtype, dev, "workspace"), workspace


def add_rms_norm(x, weight, y=None, residual=None, h=None, q=None, scales=None, rstd=None,
                 eps=1e-6, stream=None):
    """h = x + residual (out, the new residual stream; without a residual h is x
    and is not given); y (out) = h / rms(h) * weight, and / or the same in E4M3:
    q (out, uint8 / float8_e4m3fn [rows, K]) with scales (out) fp32 [rows,
    ceil(K / 128)] or, one for each row, [rows].  rstd (out, fp32 [rows]) is
    1 / rms, for the gradient.  x, residual, h, y [rows, K] and weight [K] of one
    type, bf16 / fp16 / fp32; h and y may be x or residual themselves."""
    p, xs, dev = _matrix(x, "x")
    shape = x.shape
    n, k = shape
    dt = x.dtype
    pr, rs = None, k
    if residual is not None:
        pr, rs, _ = _matrix(residual, "residual", dt, shape, dev)
    f32 = torch.float32
    pw = _array(weight, (k,), dt, dev, "weight")
    ph = None if h is None else _array(h, shape, dt, dev, "h")
    py = None if y is None else _array(y, shape, dt, dev, "y")
    pq = None if q is None else _array_of(q, shape, _U8, dev, "q")
    by_row, ps = False, None
    if scales is not None:
        by_row = scales.dim() == 1
        ps = _array(scales, (n,) if by_row else (n, _blocks128(k)), f32, dev, "scales")
    pu = None if rstd is None else _array(rstd, (n,), f32, dev, "rstd")
    _on_current_device(dev)
    _checked("moeq_add_rms_norm", (_lib or lib()).moeq_add_rms_norm(
        DTYPES[dt], p, xs, pr, rs, n, k, pw, eps, ph, py, pq, ps, by_row, pu, _stream(stream)))


def add_rms_norm_grad_workspace(rows, K):
    """Bytes of the workspace that add_rms_norm_grad takes for d_weight."""
    return lib().moeq_add_rms_norm_grad_workspace(rows, K)


def add_rms_norm_grad(d_y, h, weight, rstd, d_x, d_weight=None, d_h=None, workspace=None,
                      stream=None):
    """Gradient of add_rms_norm: d_x (out, x's and the residual's alike) from d_y,
    the forward call's h (x where there was no residual) and rstd, plus d_h, what
    reaches h along the residual stream; d_weight (out, fp32 [K]).  workspace:
    add_rms_norm_grad_workspace(rows, K) bytes, needed with d_weight; without
    one it is allocated, on the current stream (so give it with another)."""
    p, ys, dev = _matrix(d_y, "d_y")
    shape = d_y.shape
    n, k = shape
    dt, f32 = d_y.dtype, torch.float32
    ph, hs, _ = _matrix(h, "h", dt, shape, dev)
    pd, ds = None, k
    if d_h is not None:
        pd, ds, _ = _matrix(d_h, "d_h", dt, shape, dev)
    pw = _array(weight, (k,), dt, dev, "weight")
    pu = _array(rstd, (n,), f32, dev, "rstd")
    px = _array(d_x, shape, dt, dev, "d_x")
    pg = ws = None
    if d_weight is not None:
        pg = _array(d_weight, (k,), f32, dev, "d_weight")
        ws, workspace = _workspace(workspace, add_rms_norm_grad_workspace(n, k), stream, d_y, dev)
    _on_current_device(dev)
    _checked("moeq_add_rms_norm_grad", (_lib or lib()).moeq_add_rms_norm_grad(
        DTYPES[dt], p, ys, pd, ds, ph, hs, n, k, pw, pu, px, pg, ws, _stream(stream)))


def grouped_matmul_fp8_block(c, a, b, a_scales, b_scales, a_offsets, expert_ids,
                             max_tokens_per_expert=0, num_active_experts=None, stream=None):
    """Grouped FP8 matmul with a scale for each block of 128: c bf16 [rows, N]
    (out); a [rows, K] with a_scales [rows, ceil(K / 128)]; b [E, N, K] with
    b_scales [E, ceil(N / 128), ceil(K / 128)]; group g is rows
    [a_offsets[g], a_offsets[g + 1]) of expert expert_ids[g]."""
    G = expert_ids.numel() if num_active_experts is None else num_active_experts
    E, N, K = b.shape
    if expert_ids.numel() < G or a_offsets.numel() < G + 1:
        raise ValueError(f"a_offsets, expert_ids: too short for {G} groups")
    T = a.shape[0]
    _call("moeq_grouped_matmul_fp8_block", _shaped(c, (T, N), torch.bfloat16, "c"),
          _shaped(a, (T, K), _U8, "a"), _ptr(b, _U8, "b"),
          _shaped(a_scales, (T, _blocks128(K)), torch.float32, "a_scales"),
          _shaped(b_scales, (E, _blocks128(N), _blocks128(K)), torch.float32,
                  "b_scales"),
          _ptr(a_offsets, _U32, "a_offsets"), _ptr(expert_ids, torch.int32, "expert_ids"), T, N, K,
          E, max_tokens_per_expert, G, _stream(stream))


def grouped_matmul_fp8_block_epilogue(c, a, b, a_scales, b_scales, a_offsets, expert_ids,
                                      bias=None, activation=None, residual=None, z=None,
                                      max_tokens_per_expert=0, num_active_experts=None,
                                      stream=None):
    """grouped_matmul_fp8_block with an epilogue: c = act(product + bias of the
    row's expert) + residual, rounded once.  bias fp32 [E, N]; activation None,
    "relu", "silu", "gelu" or "gelu_tanh"; residual bf16 [rows, N] (may be c
    itself); z (out, bf16 [rows, N]) is the product with bias, for the gradient."""
    pa, _, dev = _matrix(a, "a", a.dtype)
    T, K = a.shape
    E, N, _ = b.shape
    out, bf16, f32 = (T, N), torch.bfloat16, torch.float32
    if a.dtype not in _U8:
        raise TypeError(f"a: dtype {a.dtype}, expected one of {_U8}")
    if not a.is_contiguous():
        raise ValueError("a: must be contiguous")
    ro, ids, G = _groups(a_offsets, expert_ids, num_active_experts, dev)
    pc = _array(c, out, bf16, dev, "c")
    pb = _array_of(b, (E, N, K), _U8, dev, "b")
    kb = _blocks128(K)
    psa = _array(a_scales, (T, kb), f32, dev, "a_scales")
    psb = _array(b_scales, (E, _blocks128(N), kb), f32, dev, "b_scales")
    pv = None if bias is None else _array(bias, (E, N), f32, dev, "bias")
    pr = None if residual is None else _array(residual, out, bf16, dev, "residual")
    pz = None if z is None else _array(z, out, bf16, dev, "z")
    _on_current_device(dev)
    _checked("moeq_grouped_matmul_fp8_block_epilogue",
             (_lib or lib()).moeq_grouped_matmul_fp8_block_epilogue(
                 pc, pa, pb, psa, psb, pv, _one_of(ACTIVATIONS, activation, "activation"), pr, pz,
                 ro, ids, T, N, K, E, max_tokens_per_expert, G, _stream(stream)))


def grouped_epilogue_grad_workspace(rows, N, num_active_experts):
    """Bytes of the workspace that grouped_epilogue_grad takes for d_bias."""
    return lib().moeq_grouped_epilogue_grad_workspace(rows, N, num_active_experts)


def grouped_epilogue_grad(d_c, a_offsets, expert_ids, num_experts, z=None, activation=None, q=None,
                          scales=None, d_z=None, d_bias=None, workspace=None,
                          num_active_experts=None, stream=None):
    """Gradient of grouped_matmul_fp8_block_epilogue's epilogue: d_z = d_c *
    act'(z) as q (out, uint8 / float8_e4m3fn [rows, N]) with scales (out, fp32
    [rows, ceil(N / 128)]) and / or as d_z (out, bf16), and d_bias (out, fp32
    [num_experts, N]), its sums over each expert's rows.  d_c bf16 [rows, N]; z
    as the forward call saved it, with an activation.  workspace:
    grouped_epilogue_grad_workspace(rows, N, groups) bytes, needed with d_bias;
    without one it is allocated, on the current stream (so give it with another)."""
    p, cs, dev = _matrix(d_c, "d_c", torch.bfloat16)
    shape = d_c.shape
    T, N = shape
    bf16, f32 = torch.bfloat16, torch.float32
    ro, ids, G = _groups(a_offsets, expert_ids, num_active_experts, dev)
    pz = None if z is None else _array(z, shape, bf16, dev, "z")
    pq = None if q is None else _array_of(q, shape, _U8, dev, "q")
    ps = None if scales is None else _array(scales, (T, _blocks128(N)), f32, dev, "scales")
    pd = None if d_z is None else _array(d_z, shape, bf16, dev, "d_z")
    pv = ws = None
    if d_bias is not None:
        pv = _array(d_bias, (num_experts, N), f32, dev, "d_bias")
        ws, workspace = _workspace(workspace, grouped_epilogue_grad_workspace(T, N, G), stream,
                                   d_c, dev)
    _on_current_device(dev)
    _checked("moeq_grouped_epilogue_grad", (_lib or lib()).moeq_grouped_epilogue_grad(
        p, cs, pz, _one_of(ACTIVATIONS, activation, "activation"), pq, ps, pd, pv, ro, ids, T, N,
        num_experts, G, ws, _stream(stream)))


def get_device_error(stream=None):
    """Sticky device error bits (synchronises the stream)."""
    v = ctypes.c_uint32(0)
    st = lib().moeq_get_device_error(_stream(stream), ctypes.byref(v))
    if st not in (0, 4):
        raise MoeqError("moeq_get_device_error", st)
    return v.value


def clear_device_error(stream=None):
    _call("moeq_clear_device_error", _stream(stream))


def sf_bytes(rows, kv):
    """Bytes of a tiled block-scale buffer for [rows, kv] logical scales."""
    return (rows + 127) // 128 * ((kv + 3) // 4) * 512
