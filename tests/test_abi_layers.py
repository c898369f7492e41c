"""Refusals of the scored router, norm and epilogue calls: bad host arguments
return their status before anything is launched (no GPU, no compute call)."""
import torch

import pytest

from fp4_fp8_quantization_gb300 import moeq
from tests.test_abi_experts import BAD, FAKE, ODD, OK, UNSUPPORTED, _caller, lib  # noqa: F401


def test_gate_group_refusals(lib):  # noqa: F811
    call = _caller(lib.moeq_gate_group_topk, dict(
        dt=0, x=FAKE, stride=64, T=8, E=64, b=FAKE, score=1, G=8, some=2, gs=1, k=4, norm=1, s=1.0,
        ids=FAKE, w=FAKE, st=None))
    assert call(dt=3) == BAD and call(T=-1) == BAD and call(E=0) == BAD and call(stride=63) == BAD
    assert call(score=2) == BAD and call(score=-1) == BAD and call(gs=2) == BAD
    assert call(G=0) == BAD and call(G=7) == BAD and call(G=-8) == BAD
    assert call(some=0) == BAD and call(some=9) == BAD and call(k=0) == BAD
    assert call(some=2, k=17) == BAD                       # more than the kept experts
    assert call(x=None) == BAD and call(x=ODD) == BAD and call(b=ODD) == BAD
    assert call(ids=None) == BAD and call(w=ODD) == BAD
    assert call(E=1025, stride=1025, G=1, some=1) == UNSUPPORTED
    assert call(G=1, some=1, k=33) == UNSUPPORTED
    assert call(G=64, some=64) == UNSUPPORTED
    assert call(E=1023, stride=1023, G=3) == UNSUPPORTED   # 341 experts on 8 lanes
    assert call(T=1 << 30) == UNSUPPORTED
    assert call(T=0, x=None, b=None, ids=None, w=None) == OK


def test_gate_group_grad_refusals(lib):  # noqa: F811
    call = _caller(lib.moeq_gate_group_topk_grad, dict(
        dt=0, x=FAKE, stride=64, T=8, E=64, score=1, k=4, norm=1, s=1.0, ids=FAKE, dw=FAKE,
        dx=FAKE, st=None))
    for score in (0, 1):
        assert call(score=score, dt=3) == BAD and call(score=score, T=-1) == BAD
        assert call(score=score, k=65) == BAD and call(score=score, stride=63) == BAD
        for p in ("x", "ids", "dw", "dx"):
            assert call(**{"score": score, p: None}) == BAD
            assert call(**{"score": score, p: ODD}) == BAD
        assert call(score=score, k=33) == UNSUPPORTED
        assert call(score=score, T=0, x=None, ids=None, dw=None, dx=None) == OK
    assert call(score=2) == BAD


def test_binding_refuses_host_tensors():
    x, ids = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        moeq.gate_group_topk(x, ids, torch.zeros(4, 2))
    with pytest.raises(ValueError):
        moeq.gate_group_topk_grad(x, ids, torch.zeros(4, 2), x)


def test_norm_refusals(lib):  # noqa: F811
    call = _caller(lib.moeq_add_rms_norm, dict(
        dt=0, x=FAKE, xs=64, r=FAKE, rs=64, R=8, K=64, w=FAKE, eps=1e-6, h=FAKE, y=0x20000, q=FAKE,
        s=FAKE, by_row=0, u=FAKE, st=None))
    assert call(y=FAKE) == BAD                             # h itself
    assert call(dt=3) == BAD and call(R=-1) == BAD and call(K=0) == BAD and call(K=68, xs=72, rs=72) == BAD
    assert call(K=56) == BAD                               # codes of a K that is no multiple of 16
    assert call(eps=-1.0) == BAD and call(eps=float("nan")) == BAD
    assert call(xs=56) == BAD and call(xs=68) == BAD and call(rs=60) == BAD
    for p in ("x", "r", "w", "h", "y", "q", "s", "u"):
        assert call(**{p: ODD}) == BAD
    for p in ("x", "w", "h", "q", "s", "r"):               # h goes with a residual, scales with codes
        assert call(**{p: None}) == BAD
    assert call(y=None, q=None, s=None, u=None) == BAD     # nothing to compute
    assert call(K=16392, xs=16392, rs=16392) == UNSUPPORTED and call(R=1 << 31) == UNSUPPORTED
    assert call(R=0, x=None, w=None, r=None, h=None) == OK


def test_norm_grad_refusals(lib):  # noqa: F811
    call = _caller(lib.moeq_add_rms_norm_grad, dict(
        dt=0, dy=FAKE, dys=64, dh=FAKE, dhs=64, h=FAKE, hs=64, R=8, K=64, w=FAKE, u=FAKE, dx=FAKE,
        dw=FAKE, ws=FAKE, st=None))
    assert call(dt=3) == BAD and call(R=-1) == BAD and call(K=0) == BAD and call(K=60) == BAD
    for p in ("dy", "dh", "h", "w", "u", "dx", "dw", "ws"):
        assert call(**{p: ODD}) == BAD
    for p in ("dy", "h", "w", "u", "dx", "ws"):
        assert call(**{p: None}) == BAD
    for p in ("dys", "dhs", "hs"):
        assert call(**{p: 56}) == BAD and call(**{p: 68}) == BAD
    assert call(K=16392, dys=16392, dhs=16392, hs=16392) == UNSUPPORTED
    assert call(R=0, dw=None, dy=None, h=None, w=None, u=None, dx=None, ws=None) == OK
    size = lib.moeq_add_rms_norm_grad_workspace
    assert size(-1, 64) == -1 and size(8, 60) == -1 and size(8, 1 << 20) == -1
    assert size(0, 64) == 0 and size(1, 4096) == 4096 * 4 and size(1 << 30, 4096) == 304 * 4096 * 4


def test_norm_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        moeq.add_rms_norm(x, x[0], y=x)
    with pytest.raises(ValueError):
        moeq.add_rms_norm_grad(x, x, x[0], x[:, 0], x)


def test_epilogue_gemm_refusals(lib):  # noqa: F811
    call = _caller(lib.moeq_grouped_matmul_fp8_block_epilogue, dict(
        c=FAKE, a=FAKE, b=FAKE, sa=FAKE, sb=FAKE, bias=FAKE, act=2, res=FAKE, z=0x20000, ro=FAKE,
        ids=FAKE, T=64, N=72, K=144, E=2, mt=8, G=2, st=None))
    assert call(K=136) == BAD and call(N=68) == BAD and call(K=0) == BAD and call(T=-1) == BAD
    assert call(E=0) == BAD and call(G=-1) == BAD and call(ro=None) == BAD and call(ids=None) == BAD
    assert call(act=5) == BAD and call(act=-1) == BAD
    for p in ("c", "a", "b", "sa", "sb"):
        assert call(**{p: None}) == BAD
    for p in ("c", "a", "b", "sa", "sb", "bias", "res", "z"):
        assert call(**{p: ODD}) == BAD
    assert call(z=FAKE) == BAD                             # c itself
    assert call(G=1025) == UNSUPPORTED and call(T=1 << 31) == UNSUPPORTED
    assert call(G=0) == OK and call(T=0, a=None, c=None, sa=None, res=None, z=None) == OK


def test_epilogue_grad_refusals(lib):  # noqa: F811
    call = _caller(lib.moeq_grouped_epilogue_grad, dict(
        dc=FAKE, dcs=64, z=FAKE, act=2, q=FAKE, s=FAKE, dz=FAKE, db=FAKE, ro=FAKE, ids=FAKE, T=8,
        N=64, E=2, G=2, ws=FAKE, st=None))
    assert call(T=-1) == BAD and call(N=0) == BAD and call(N=68) == BAD and call(E=0) == BAD
    assert call(N=56) == BAD                               # codes of an N that is no multiple of 16
    assert call(dcs=56) == BAD and call(dcs=68) == BAD and call(act=5) == BAD and call(act=-1) == BAD
    for p in ("dc", "z", "q", "s", "dz", "db", "ws"):
        assert call(**{p: ODD}) == BAD
    for p in ("dc", "z", "q", "s", "ws", "ro", "ids"):
        assert call(**{p: None}) == BAD
    assert call(act=0) == BAD                              # z without an activation
    assert call(q=None, s=None, dz=None, db=None) == BAD   # nothing to compute
    assert call(G=1025) == UNSUPPORTED and call(T=1 << 31) == UNSUPPORTED and call(E=65536) == UNSUPPORTED
    assert call(T=0, db=None, dc=None, z=None, q=None, s=None) == OK
    size = lib.moeq_grouped_epilogue_grad_workspace
    assert size(-1, 64, 2) == -1 and size(8, 60, 2) == -1 and size(8, 64, 1025) == -1
    assert size(8, 64, 2) == 16 + 2 * 64 * 4 and size(1000, 64, 3) == 16 + (15 + 3) * 64 * 4
    assert size(1 << 20, 64, 3) == 16 + (4096 + 3) * 64 * 4
    assert size(0, 64, 4) == 32


def test_epilogue_binding_refuses_host_tensors():
    x, ids = torch.zeros(4, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        moeq.grouped_matmul_fp8_block_epilogue(x, x, torch.zeros(1, 8, 64), x, x, ids, ids[:1])
    with pytest.raises(ValueError):
        moeq.grouped_epilogue_grad(x.bfloat16(), ids, ids[:1], 1, d_z=x)
