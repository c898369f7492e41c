"""The scored router's choice where what is close together is not next to one another
in the order that fp32 values and shortened keys give, against the float64 oracle."""
import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq
from tests._util import need_gpu
from tests.test_gpu_gate_group import _gate, _want

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _error_word():
    need_gpu()
    moeq.clear_device_error()
    yield
    assert moeq.get_device_error() == 0


def _same_choice(x, k, bias, **kw):
    """Few tokens, and the same ones among many."""
    x, bias = torch.from_numpy(x), torch.from_numpy(bias)
    want, _ = _want(x, k, bias, **kw)
    for reps in (1, -(-4200 // len(x)), -(-8300 // len(x))):
        ids, _ = _gate(x.repeat(reps, 1), k, bias, **kw)
        got = ids.cpu().numpy().reshape(reps, len(x), k)
        assert (got == got[:1]).all()
        wrong = (got[0] != want).any(1)
        assert not wrong.any(), (int(wrong.sum()), got[0][wrong][0], want[wrong][0])


def _logit(s):
    """fp32 logits whose sigmoid is s, to their rounding."""
    return np.log(s / (1.0 - s)).astype(np.float32)


def test_a_left_over_value_as_good_as_a_choice_that_is_not_the_last():
    """One expert far above, so that the distances from it are coarse in steps of 2^-17
    (half of them, 0.15, as fp32 with 8 bits left to the index).  At the border of two
    steps lie a: just above it, b: above it, of a higher index than a; c: below it, d: a
    few 2^-30 above a, but where fp32 rounds it down to the border.  The better of a and
    d is a choice, and b is another one."""
    rng = np.random.default_rng(1)
    T, E, k = 600, 256, 8
    a, b, c, d = 40, 90, 150, 200
    bias = np.zeros(E, np.float32)
    bias[1:] = rng.uniform(-0.1, 0.1, E - 1).astype(np.float32)
    border = 1.0 - rng.integers(round(0.27 * 2 ** 17), round(0.33 * 2 ** 17), T) * 2.0 ** -17
    value = np.empty((T, E))
    value[:] = border[:, None] - rng.uniform(0.05, 0.15, (T, E))
    value[:, 10:15] = border[:, None] + 0.01 * np.arange(1, 6)
    value[:, b] = border + 4e-6
    value[:, c] = border - 2e-6
    half = 2.0 ** -25                                      # of a unit of values in [0.5, 1)
    value[:, a] = border + half + rng.uniform(-1, 1, T) * 2.0 ** -28
    value[:, d] = value[:, a] + rng.uniform(0, 1, T) * 2.0 ** -28
    x = _logit(value - bias)
    x[:, 0] = 40.0                                         # 1 to the last bit of fp32
    _same_choice(x, k, bias)
