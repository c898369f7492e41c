"""Buffers that a call may not write over one another are refused before anything is
launched (no GPU, no compute call)."""
from tests.test_abi_experts import BAD, FAKE, OK, _caller, lib  # noqa: F401


def test_scored_router_gradient_over_its_logits(lib):  # noqa: F811
    """The gradient of the chosen logits zeroes a row before it reads them."""
    call = _caller(lib.moeq_gate_group_topk_grad, dict(
        dt=0, x=FAKE, stride=64, T=8, E=64, score=1, k=4, norm=1, s=1.0, ids=0x20000, dw=0x30000,
        dx=FAKE, st=None))
    for score, norm in ((1, 0), (1, 1), (0, 1)):
        assert call(score=score, norm=norm) == BAD
        assert call(score=score, norm=norm, T=0) == OK
