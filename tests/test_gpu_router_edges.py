"""The router's weights at the edges of its definition."""
import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq
from oracle import experts as X
from tests._util import DEV, need_gpu
from tests.test_gpu_experts import _gate

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("normalize", [False, True])
def test_nan_reaches_the_places_left_over(normalize, dtype):
    """A token with a NaN and fewer choices than places: no id for the rest, and
    every weight of the token is NaN; without any choice they are 0."""
    need_gpu()
    moeq.clear_device_error()
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[nan, 1.0, -inf, -inf], [inf, -inf, -inf, -inf], [nan, -inf, nan, -inf],
                      [nan] * 4, [-inf, 2.0, -inf, 0.5]], dtype=dtype)
    ids, w = _gate(x.to(DEV), 3, normalize, 2.0)
    want_ids, want_w = X.gate_topk(x.double().numpy(), 3, normalize, 2.0)
    assert ids.tolist() == want_ids.tolist() == [[1, -1, -1], [0, -1, -1], [-1] * 3, [-1] * 3,
                                                 [1, 3, -1]]
    assert torch.isnan(w[:2]).all() and not w[2:4].any()
    assert np.isnan(want_w[:2]).all() and not want_w[2:4].any()
    assert np.allclose(w[4].cpu().numpy(), want_w[4], rtol=1e-6, atol=0)
    assert moeq.get_device_error() == 0


@pytest.mark.parametrize("E", [4, 40, 200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("normalize", [False, True])
def test_gradient_of_tokens_with_nan_or_infinity(normalize, dtype, E):
    need_gpu()
    moeq.clear_device_error()
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(5, E)
    x[0, E - 1] = nan
    x[1, 1] = inf
    x[2] = -inf
    x[2, 0] = nan                       # nothing to choose
    x[3] = -inf
    x[3, 2] = 1.0                       # a single choice: weight 1, nothing to learn
    x[4, 1] = -inf
    x = x.to(dtype).to(DEV)
    ids, _ = _gate(x, 3, normalize, 1.0)
    dx = torch.full_like(x, 7.0)
    dw = torch.tensor([1.0, -2.0, 0.5], device=DEV).expand(5, 3).contiguous()
    moeq.gate_topk_grad(x, ids, dw, dx, normalize=normalize)
    chosen = torch.zeros(5, E, dtype=torch.bool, device=DEV)
    for t in range(5):
        chosen[t, ids[t][ids[t] >= 0].long()] = True
    if normalize:
        assert torch.isnan(dx[:2][chosen[:2]]).all() and not dx[:2][~chosen[:2]].any()
    else:
        assert torch.isnan(dx[:2]).all()
    assert not dx[2:4].any()
    want = X.gate_topk_grad(x[4:].double().cpu().numpy(), ids[4:].cpu().numpy(),
                            dw[4:].cpu().numpy(), normalize, 1.0)
    # exp(0) = 1 and sums of ones are exact: a division, a sum of three products
    # and two products, 2^-24 each on terms of at most 2, and the rounding of dtype
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[dtype]
    err = np.abs(dx[4].double().cpu().numpy() - want[0]).max()
    assert err <= u * np.abs(want).max() + 16 * 2.0 ** -24
    assert moeq.get_device_error() == 0
