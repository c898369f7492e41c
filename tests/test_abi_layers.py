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
