"""Refusals of the router, row, FP8-block and FP8-block GEMM calls: bad host
arguments return their status before anything is launched, and the binding
raises on tensors of the wrong kind (no GPU, no compute call is made)."""
import ctypes
import os

import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq

FAKE = ctypes.c_void_p(0x10000)   # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10004)
BAD, UNSUPPORTED, OK = 1, 2, 0


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moeq._LIB_PATH):
        from fp4_fp8_quantization_gb300 import build
        build.build()
    return moeq.lib()


def _caller(f, ok):
    def call(**kw):
        assert set(kw) <= set(ok)
        return f(*dict(ok, **kw).values())
    return call


def test_gate_refusals(lib):
    fwd = _caller(lib.moeq_gate_topk, dict(dt=0, x=FAKE, stride=64, T=8, E=64, k=4, norm=1, s=1.0,
                                           ids=FAKE, w=FAKE, st=None))
    bwd = _caller(lib.moeq_gate_topk_grad, dict(dt=0, x=FAKE, stride=64, T=8, E=64, k=4, norm=1,
                                                s=1.0, ids=FAKE, w=FAKE, dx=FAKE, st=None))
    for call in (fwd, bwd):
        assert call(dt=3) == BAD and call(dt=-1) == BAD
        assert call(T=-1) == BAD and call(k=0) == BAD and call(k=65) == BAD and call(E=0) == BAD
        assert call(stride=63) == BAD and call(x=None) == BAD and call(x=ODD) == BAD
        assert call(ids=None) == BAD and call(w=ODD) == BAD
        assert call(E=1025, stride=1025) == UNSUPPORTED and call(k=33) == UNSUPPORTED
        assert call(T=1 << 30) == UNSUPPORTED
        assert call(T=0, x=None, ids=None, w=None) == OK
    assert bwd(dx=None) == BAD


def test_row_refusals(lib):
    permute = _caller(lib.moeq_permute_topk, dict(
        dt=0, x=FAKE, stride=64, T=8, H=64, dst=FAKE, k=2, w=FAKE, rows=FAKE, R=16, st=None))
    permute_grad = _caller(lib.moeq_permute_topk_grad, dict(
        dt=0, rows=FAKE, R=16, T=8, H=64, dst=FAKE, k=2, w=FAKE, x=FAKE, tok=FAKE, stride=64,
        dw=FAKE, st=None))
    combine = _caller(lib.moeq_combine_topk, dict(
        dt=0, rows=FAKE, R=16, T=8, H=64, dst=FAKE, k=2, w=FAKE, x=FAKE, st=None))
    combine_grad = _caller(lib.moeq_combine_topk_grad, dict(
        dt=0, x=FAKE, stride=64, T=8, H=64, dst=FAKE, k=2, w=FAKE, d_rows=FAKE, R=16, rows=FAKE,
        dw=FAKE, st=None))
    for call in (permute, permute_grad, combine, combine_grad):
        assert call(dt=7) == BAD and call(T=-1) == BAD and call(k=0) == BAD and call(R=-1) == BAD
        assert call(H=0) == BAD and call(H=60) == BAD          # 120-byte rows
        assert call(dst=None) == BAD and call(dst=ODD) == BAD and call(w=ODD) == BAD
        assert call(x=None) == BAD and call(x=ODD) == BAD and call(rows=ODD) == BAD
        assert call(k=33) == UNSUPPORTED and call(R=1 << 31) == UNSUPPORTED
        assert call(T=1 << 30) == UNSUPPORTED
        assert call(T=0, x=None, rows=None, dst=None) == OK
    assert permute(rows=None) == BAD and combine(rows=None) == BAD
    for call in (permute, permute_grad, combine_grad):
        assert call(stride=56) == BAD and call(stride=68) == BAD
    assert permute_grad(tok=None) == BAD                       # d_weights without tokens
    assert combine_grad(rows=None) == BAD                      # d_weights without rows
    assert combine_grad(d_rows=None) == BAD and combine_grad(dw=ODD) == BAD


def test_fp8_block_refusals(lib):
    rows = _caller(lib.moeq_quantize_fp8_block, dict(x=FAKE, stride=160, R=8, K=160, q=FAKE,
                                                     s=FAKE, st=None))
    topk = _caller(lib.moeq_quantize_fp8_block_topk, dict(
        x=FAKE, stride=160, R=8, K=160, dst=FAKE, k=2, q=FAKE, s=FAKE, n=16, st=None))
    swiglu = _caller(lib.moeq_swiglu_quantize_fp8_block, dict(x=FAKE, R=8, K=160, q=FAKE, s=FAKE,
                                                              st=None))
    weight = _caller(lib.moeq_quantize_fp8_block_weight, dict(x=FAKE, E=2, R=8, K=160, q=FAKE,
                                                              s=FAKE, st=None))
    for call in (rows, topk, swiglu, weight):
        assert call(K=0) == BAD and call(K=168) == BAD and call(R=-1) == BAD
        assert call(x=None) == BAD and call(x=ODD) == BAD and call(q=ODD) == BAD
        assert call(s=None) == BAD and call(q=None) == BAD
        assert call(R=0, x=None, q=None, s=None) == OK
    for call in (rows, topk):
        assert call(stride=152) == BAD and call(stride=164) == BAD
    assert topk(k=0) == BAD and topk(dst=None) == BAD and topk(k=33) == UNSUPPORTED
    assert weight(E=-1) == BAD and weight(E=70000) == UNSUPPORTED


def test_fp8_block_gemm_refusals(lib):
    call = _caller(lib.moeq_grouped_matmul_fp8_block, dict(
        c=FAKE, a=FAKE, b=FAKE, sa=FAKE, sb=FAKE, ro=FAKE, ids=FAKE, T=64, N=72, K=144, E=2, mt=8,
        G=2, st=None))
    assert call(K=136) == BAD and call(N=68) == BAD and call(K=0) == BAD and call(T=-1) == BAD
    assert call(E=0) == BAD and call(G=-1) == BAD and call(ro=None) == BAD and call(ids=None) == BAD
    for p in ("c", "a", "b", "sa", "sb"):
        assert call(**{p: None}) == BAD and call(**{p: ODD}) == BAD
    assert call(G=1025) == UNSUPPORTED and call(T=1 << 31) == UNSUPPORTED
    assert call(G=0) == OK and call(T=0, a=None, c=None, sa=None) == OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        moeq.gate_topk(x, ids, torch.zeros(4, 2))
    with pytest.raises(ValueError):
        moeq.permute_topk(x, ids, torch.zeros(8, 64))
    with pytest.raises(ValueError):
        moeq.combine_topk(torch.zeros(8, 64), ids, x)
    with pytest.raises(ValueError):
        moeq.quantize_fp8_block(x.bfloat16(), x, x)
    with pytest.raises(ValueError):
        moeq.grouped_matmul_fp8_block(x, x, torch.zeros(2, 8, 64), x, x, ids, ids)
