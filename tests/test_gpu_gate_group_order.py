"""The scored router's choice where what is close together is not next to one another
in the order that fp32 values and shortened keys give, against the float64 oracle."""
import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq
from oracle import layers as L
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


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,size,some", [(3, 2, 1), (8, 2, 4), (8, 4, 3), (16, 2, 5), (5, 3, 2)])
def test_group_sums_that_cancel(G, size, some, score):
    """The best two of a group cancel to the rounding of values far larger: it may be
    better than groups that are not next to it in the order of fp32 sums."""
    rng = np.random.default_rng(G * size)
    T, E = 300, G * size
    large = rng.choice([0.0, 100.0, 1000.0, 10000.0], G)
    large[:3] = 0.0, 0.0, 1000.0
    bias = np.full((G, size), -2e4, np.float32)            # what is behind the best two
    bias[:, 0], bias[:, 1] = large, -large
    spread = np.where(rng.random(T) < 0.5, 1e-5, 1e-3)[:, None]
    if score == "sigmoid":
        x = 0.2 + rng.normal(size=(T, E)) * spread
    else:
        x = rng.normal(size=(T, E)) * spread * 10
    x[0] = 0.0
    bias[0, 1], bias[1, 1] = 4e-5, 2e-5
    x[0, 2 * size:2 * size + 2] = 1.1e-4
    # Where there are more than three groups, the first row's others have the same scores, and
    # (s + large) + (s - large) is 2 s in the reals for each of them: equal but for the rounding
    # of 64 bits, which may fall either way.  The row is compared where there are three.
    x = x[G > 3:].astype(np.float32)
    for k in (1, min(8, some * size)):
        _same_choice(x, k, bias.reshape(-1), num_groups=G, topk_groups=some, score=score)


def test_the_first_group_of_large_values_in_64_bits():
    """Sums 1.00004, 1.00002 and 1.000055, the last of 1000.5 and -999.5."""
    x = np.float32([[0, 0, 0, 0, 1.1e-4, 1.1e-4]])
    bias = np.float32([0, 4e-5, 0, 2e-5, 1000, -1000])
    assert L.gate_group_topk(x, 1, bias, groups=3, topk_groups=1)[0].tolist() == [[4]]
    _same_choice(x, 1, bias, num_groups=3, topk_groups=1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_group_sums_past_the_range_of_fp32(score):
    """Biases of the type's lowest and largest value: -6.8e38 is above a group without an
    expert, and 6.8e38 above 5e38."""
    low, inf = float(np.finfo(np.float32).min), float("inf")
    rng = np.random.default_rng(2)
    T = 40
    for values in ([(None, None), (low, low), (0, 0), (None, None)],
                   [(None, None), (None, low), (low, low), (0, low)],
                   [(2.5e38, 2.5e38), (-low, -low), (0, 0), (3e38, 1.5e38)],
                   [(low, low), (low, low), (-low, low), (2.0, -2.0)],
                   [(inf, 0.0), (-low, -low), (inf, 1.0), (low, low)]):
        x = rng.normal(size=(T, 4, 3)).astype(np.float32)
        bias = np.full((4, 3), low, np.float32)
        x[:, :, 2] = -inf
        for g, pair in enumerate(values):
            for j, v in enumerate(pair):
                if v is None:
                    x[:, g, j] = -inf
                else:
                    bias[g, j] = v
        for some in (1, 2, 3):
            for k in (1, 3):
                _same_choice(x.reshape(T, 12), k, bias.reshape(-1), num_groups=4, topk_groups=some, score=score)
