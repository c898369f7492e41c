"""The router with scores, a balance bias and groups on the GPU against the
float64 oracle.

The choice is the order of 64-bit values and is compared for equality.
Weights: sigmoid(x) is within 2 ulp of its exp (|relative| 2^-22 (1 - s)), a
sum and a quotient, below 4 2^-24; normalised, the sum of k of them and one
more quotient, k 2^-24.  Softmax as for the plain router: exp(d) within 2 +
1.173 |d| ulp of 2^-23, its argument within |d| 2^-24, sums of E terms within
(E / 32 + 6) 2^-24.  u(dtype) is half a unit in the last place.
"""
import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq
from oracle import layers as L
from tests._util import DEV, need_gpu
from tests.test_gpu_experts import DTYPES, EPS, TINY, U, close, f64
from tests.test_gpu_guard_regions import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _error_word():
    need_gpu()
    moeq.clear_device_error()
    yield
    assert moeq.get_device_error() == 0


def _gate(x, k, bias=None, guard=None, **kw):
    T = x.shape[0]
    new = guard or (lambda s, d: torch.full(s, -9, dtype=d, device=DEV))
    ids, w = new((T, k), torch.int32), new((T, k), torch.float32)
    moeq.gate_group_topk(x.to(DEV), ids, w, bias=None if bias is None else bias.to(DEV), **kw)
    return ids, w


def _want(x, k, bias=None, num_groups=1, **kw):
    return L.gate_group_topk(f64(x), k, None if bias is None else f64(bias), groups=num_groups, **kw)


def _rel(x, k, score):
    """Relative error of the weights."""
    if score == "sigmoid":
        return np.full((x.shape[0], 1), (10 + k) * EPS)
    spread = np.nan_to_num(x, neginf=0).max(1) - np.where(np.isfinite(x), x, np.inf).min(1)
    spread = np.minimum(np.abs(np.nan_to_num(spread)), 104.0)
    return (2.0 ** -21 + 3.5 * spread * EPS + (x.shape[1] / 32 + 10) * EPS)[:, None]


def _check(x, k, bias=None, **kw):
    ids, w = _gate(x, k, bias, **kw)
    ref_ids, ref_w = _want(x, k, bias, **kw)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    # scores below 2^-126 have fewer bits
    close(w, ref_w, _rel(f64(x), k, kw.get("score", "sigmoid")) * ref_w + 2.0 ** -120)
    return ids, w


SHAPES = [(1, 1, 1, 1, 1), (3, 6, 3, 2, 4), (33, 64, 8, 4, 6), (17, 160, 8, 3, 6), (64, 256, 8, 4, 8),
          (9, 510, 3, 2, 10), (7, 512, 16, 5, 32), (5, 1024, 1, 1, 32), (4, 1024, 32, 7, 8),
          (6, 96, 32, 32, 8), (8, 100, 1, 1, 9), (5, 20, 20, 9, 9), (2, 35, 5, 1, 7)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,G,some,k", SHAPES)
def test_choice_weights_and_gradient(T, E, G, some, k, score, dtype):
    rng = np.random.default_rng(T * E + G)
    x = torch.from_numpy(rng.normal(size=(T, E)) * 1.5).to(dtype)
    if E >= 4 * k:
        x[::3, 1::4] = float("-inf")
    bias = torch.from_numpy(rng.normal(size=E) * (0.1 if score == "sigmoid" else 1.0 / E)).float()
    for b in (None, bias, torch.zeros(E)):
        for group_score in ("top2", "max"):
            for normalize in (True, False):
                kw = dict(num_groups=G, topk_groups=some, score=score, group_score=group_score,
                          normalize=normalize, scale=2.5 if normalize else 1.0)
                ids, _ = _check(x, k, b, **kw)
    kw = dict(score=score, normalize=normalize, scale=2.5)
    for normalize in (True, False):
        kw["normalize"] = normalize
        dw = torch.from_numpy(rng.normal(size=(T, k))).float()
        dx = torch.full((T, E), 9.0, dtype=dtype, device=DEV)
        moeq.gate_group_topk_grad(x.to(DEV), ids, dw.to(DEV), dx, **kw)
        ref = L.gate_group_topk_grad(f64(x), ids.cpu().numpy(), f64(dw), score, normalize, 2.5)
        # every term is a product of weights and d_w's, each within rel; three of them meet
        size = np.abs(f64(dw)).max(1, keepdims=True) * 2.5
        rel = _rel(f64(x), k, score)
        close(dx, ref, 4 * (rel + 8 * EPS) * size + U[dtype] * np.abs(ref) + TINY[dtype])


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradient_against_differences(score, normalize):
    """The weights of fixed choices at x + h and x - h, in 64 bits."""
    rng = np.random.default_rng(3)
    T, E, k, h = 4, 12, 3, 1e-4
    x = rng.normal(size=(T, E)).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    dw = rng.normal(size=(T, k)).astype(np.float32)

    def loss(v):
        s = L.scores(v, score)
        w = np.take_along_axis(s, ids, 1)
        w = w / w.sum(1, keepdims=True) if normalize else w
        return 1.5 * (w * dw).sum(1)

    dx = torch.empty(T, E, device=DEV)
    moeq.gate_group_topk_grad(torch.from_numpy(x).to(DEV), torch.from_numpy(ids).to(DEV),
                              torch.from_numpy(dw).to(DEV), dx, score=score, normalize=normalize,
                              scale=1.5)
    for j in range(E):
        step = np.zeros((T, E))
        step[:, j] = h
        diff = (loss(x.astype(np.float64) + step) - loss(x.astype(np.float64) - step)) / (2 * h)
        # h^2 / 6 of third derivatives (below 4 |dw| here), and fp32
        assert np.all(np.abs(f64(dx)[:, j] - diff) < 1e-7 + 1e-6 * np.abs(dw).max())


@pytest.mark.parametrize("E,G,k", [(256, 8, 8), (128, 1, 8), (1024, 4, 16), (510, 3, 5), (512, 4, 32)])
def test_order_of_values_that_fp32_does_not_tell_apart(E, G, k):
    """Biases that cancel the scores' differences to a few 2^-26, equal values
    among them: the choice is that of 64 bits."""
    rng = np.random.default_rng(E)
    T = 48
    x = rng.normal(size=(1, E)).astype(np.float32)
    s = L.scores(x, "sigmoid")[0]
    bias = (1.25 - s).astype(np.float32)                  # c = 1.25 up to fp32's rounding
    x = np.repeat(x, T, 0)
    x[1::2, 3 * E // 4:] += np.float32(2.0 ** -20)        # some rows differ a little
    x[2::3, ::7] = x[2::3, :1]
    for group_score in ("max", "top2"):
        _check(torch.from_numpy(x), k, torch.from_numpy(bias), num_groups=G, topk_groups=max(1, G // 2),
               group_score=group_score)
    x[:] = x[:, :1]                                       # one value everywhere: by index
    for b in (None, torch.full((E,), 0.5)):
        for score in ("sigmoid", "softmax"):
            ids, _ = _check(torch.from_numpy(x), k, b, num_groups=G, topk_groups=1, score=score)
            assert np.array_equal(ids.cpu().numpy(), np.tile(np.arange(k), (T, 1)))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [5, 9001])
def test_many_tokens_with_ties(T, score):
    """Logits of few values: ties at every border; as few tokens and as many."""
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.integers(-3, 4, size=(5, 72)) / 2).float().bfloat16()
    bias = torch.from_numpy(rng.integers(-1, 2, size=72) / 64).float()
    for b in (None, bias):
        kw = dict(num_groups=6, topk_groups=2, score=score)
        ref, _ = _want(x, 8, b, **kw)
        ids, _ = _gate(x.repeat((T + 4) // 5, 1)[:T], 8, b, **kw)
        assert np.array_equal(ids.cpu().numpy(), np.tile(ref, ((T + 4) // 5, 1))[:T])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,some,k", [(256, 8, 4, 8), (64, 1, 1, 4), (160, 8, 3, 6), (512, 16, 5, 12),
                                        (128, 4, 2, 16), (40, 2, 1, 3), (256, 1, 1, 8), (250, 5, 3, 9),
                                        (32, 8, 8, 8), (1024, 32, 9, 17), (9, 1, 1, 2)])
def test_many_tokens_against_oracle(E, G, some, k, score, dtype):
    """Fewer lanes for each of many tokens: 47 rows, over and over."""
    rng = np.random.default_rng(E + k)
    n, T = 47, 20001
    x = torch.from_numpy(rng.normal(size=(n, E)) * 1.5).to(dtype)
    x[::5, 2::3] = float("-inf")
    x[1, 3], x[2, 4] = float("nan"), float("inf")
    x[3] = x[3, 0]
    bias = torch.from_numpy(rng.normal(size=E) * (0.1 if score == "sigmoid" else 1.0 / E)).float()
    many = x.repeat((T + n - 1) // n, 1)[:T].to(DEV)
    for b in (None, bias):
        for group_score in ("top2", "max"):
            kw = dict(num_groups=G, topk_groups=some, score=score, group_score=group_score)
            ids, w = _gate(many, k, b, **kw)
            ref_ids, ref_w = _want(x, k, b, **kw)
            for a in range(0, T, n):
                m = min(n, T - a)
                assert torch.equal(ids[a:a + m], ids[:m])
                assert torch.equal(w[a:a + m].view(torch.int32), w[:m].view(torch.int32))
            assert np.array_equal(ids[:n].cpu().numpy(), ref_ids)
            got, nan = f64(w[:n]), np.isnan(ref_w)
            assert np.array_equal(np.isnan(got), nan)
            ref_w = np.where(nan, 0.0, ref_w)
            rows = np.where(np.isfinite(f64(x)), f64(x), -np.inf)
            assert np.all(np.abs(np.where(nan, 0.0, got) - ref_w)
                          <= _rel(rows, k, score) * ref_w + 2.0 ** -120)


@pytest.mark.parametrize("E,G,k", [(256, 8, 8), (128, 1, 8), (512, 4, 16)])
def test_many_tokens_that_fp32_does_not_decide(E, G, k):
    """As above, a few such tokens among many, and all of them."""
    rng = np.random.default_rng(E + 1)
    x = rng.normal(size=(1, E)).astype(np.float32)
    bias = (1.25 - L.scores(x, "sigmoid")[0]).astype(np.float32)
    rows = np.concatenate([x, rng.normal(size=(29, E)).astype(np.float32)])
    kw = dict(num_groups=G, topk_groups=max(1, G // 2))
    ref, _ = _want(torch.from_numpy(rows), k, torch.from_numpy(bias), **kw)
    for n in (1, 30):
        many = torch.from_numpy(rows[:n]).repeat(18000 // n, 1)
        ids, _ = _gate(many, k, torch.from_numpy(bias), **kw)
        assert np.array_equal(ids.cpu().numpy(), np.tile(ref[:n], (18000 // n, 1)))


def test_rows_without_choices_and_values_that_are_none():
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(torch.float32).min
    x = torch.tensor([[-inf] * 40, [-inf] * 39 + [1.0], [nan] + [0.0] * 39, [nan] * 40,
                      [inf] + [0.0] * 39, [-0.0, 0.0] * 20, [low] * 40, [low, 1.0] * 20,
                      [-inf] * 20 + [0.5] * 20, [inf, inf, -inf, nan] * 10, [-200.0, -90.0] * 20])
    bias = torch.linspace(-0.2, 0.2, 40)
    odd = bias.clone()
    odd[3], odd[5], odd[20], odd[31] = -inf, nan, inf, -1e30
    for score in ("sigmoid", "softmax"):
        for normalize in (False, True):
            for b in (None, bias, odd):
                for G, some in ((1, 1), (4, 2), (8, 1)):
                    kw = dict(num_groups=G, topk_groups=some, score=score, normalize=normalize)
                    ids, w = _gate(x, 3, b, **kw)
                    want_ids, want_w = _want(x, 3, b, **kw)
                    assert np.array_equal(ids.cpu().numpy(), want_ids), (score, G, b)
                    assert np.allclose(f64(w), want_w, rtol=2e-6, atol=2.0 ** -120, equal_nan=True)
                    dx = torch.full_like(x, 7.0, device=DEV)
                    moeq.gate_group_topk_grad(x.to(DEV), ids, torch.ones(11, 3, device=DEV), dx,
                                              score=score, normalize=normalize)
                    assert not dx[0].any() and torch.isfinite(dx[5:9]).all()


def test_strided_rows_and_bad_ids():
    big = torch.randn(20, 136, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    for dtype in DTYPES:
        x = big.to(dtype)
        view = x[:, :64]
        one, two = _gate(view, 6, num_groups=4, topk_groups=2), None
        two = _gate(view.contiguous(), 6, num_groups=4, topk_groups=2)
        assert all(torch.equal(a, b) for a, b in zip(one, two))
        odd = x[:, :61].as_strided((20, 61), (131, 1)) if dtype == torch.float32 else x[:, :61]
        one = _gate(odd, 6)
        two = _gate(odd.contiguous(), 6)
        assert all(torch.equal(a, b) for a, b in zip(one, two))
    ids = torch.tensor([[0, 99], [-1, 3], [-7, 1]], dtype=torch.int32, device=DEV)
    x, dx = torch.zeros(3, 61, device=DEV), torch.full((3, 61), 5.0, device=DEV)
    moeq.gate_group_topk_grad(x, ids, torch.ones(3, 2, device=DEV), dx, normalize=False)
    assert moeq.get_device_error() == moeq.DEVERR_BAD_EXPERT
    moeq.clear_device_error()
    want = torch.zeros(3, 61)
    want[0, 0] = want[1, 3] = want[2, 1] = 0.25
    assert torch.equal(dx.cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,G,some,k", [(1, 1, 1, 1, 1), (5, 35, 7, 2, 9), (4101, 72, 6, 3, 5),
                                          (9, 1023, 1, 1, 32), (33, 160, 8, 8, 32)])
def test_stays_in_its_buffers(T, E, G, some, k, dtype):
    g = Guarded()
    x = torch.randn(T, E, device=DEV, generator=torch.Generator(DEV).manual_seed(2)).to(dtype)
    ids, w = _gate(x, k, torch.zeros(E), guard=g, num_groups=G, topk_groups=some)
    dx = g((T, E), dtype)
    for score in ("sigmoid", "softmax"):
        moeq.gate_group_topk_grad(x, ids, torch.ones(T, k, device=DEV), dx, score=score)
    g.check()
    assert torch.isfinite(w).all() and torch.isfinite(dx.float()).all()


def test_no_tokens():
    x = torch.empty(0, 64, device=DEV)
    ids, w = _gate(x, 4, num_groups=2, topk_groups=1)
    moeq.gate_group_topk_grad(x, ids, w, torch.empty(0, 64, device=DEV))


def test_refusals():
    x, b = torch.zeros(4, 64, device=DEV), torch.zeros(64, device=DEV)
    ids, w = torch.zeros(4, 4, dtype=torch.int32, device=DEV), torch.zeros(4, 4, device=DEV)
    for kw in (dict(score="relu"), dict(group_score="mean"), dict(bias=b[:63]), dict(bias=b.bfloat16())):
        with pytest.raises((ValueError, TypeError)):
            moeq.gate_group_topk(x, ids, w, **kw)
    for kw in (dict(num_groups=0), dict(num_groups=5), dict(num_groups=4, topk_groups=5),
               dict(num_groups=4, topk_groups=0), dict(num_groups=32, topk_groups=1),
               dict(num_groups=64)):
        with pytest.raises(moeq.MoeqError):
            moeq.gate_group_topk(x, ids, w, **kw)
    with pytest.raises(ValueError):
        moeq.gate_group_topk_grad(x, ids, w, torch.zeros(4, 63, device=DEV))
    with pytest.raises(ValueError):
        moeq.gate_group_topk(x.cpu(), ids, w)
