"""Pins of the expert-layer oracle: the gradients against central differences
of the forward definitions, the router's choice on hand-worked rows, the
E4M3 block rule on hand-worked blocks."""
import numpy as np
import pytest

from oracle import experts as X
from oracle import formats as F


def _diff(f, x, h=1e-6):
    """Gradient of the scalar f at x by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("normalize", [False, True])
def test_gate_gradient_is_the_difference_quotient(normalize):
    # third derivatives of a softmax are below 1: truncation ~h^2/6, rounding ~1e-16/h
    rng = np.random.default_rng(0)
    x = rng.permuted(np.linspace(-2, 2, 9 * 3).reshape(3, 9), axis=1)
    x[1, 4] = -np.inf
    dw = rng.normal(size=(3, 4))
    ids, _ = X.gate_topk(x, 4, normalize, 2.5)
    got = X.gate_topk_grad(x, ids, dw, normalize, 2.5)
    finite = np.isfinite(x)
    want = np.zeros_like(x)
    for i in zip(*np.nonzero(finite)):
        def f(v):
            y = x.copy()
            y[i] = v
            return float((X.gate_topk(y, 4, normalize, 2.5)[1] * dw).sum())
        want[i] = (f(x[i] + 1e-5) - f(x[i] - 1e-5)) / 2e-5
    assert np.all(got[~finite] == 0)
    assert np.abs(got - want).max() < 1e-8


def test_gate_choice_by_hand():
    n = np.nan
    x = np.array([[1, 3, 3, 2], [-np.inf, 0, -np.inf, -np.inf], [-np.inf] * 4, [n, 1, 2, n],
                  [0.0, -0.0, -1, -2]])
    ids, w = X.gate_topk(x, 3, True, 1.0)
    assert ids.tolist() == [[1, 2, 3], [1, -1, -1], [-1, -1, -1], [2, 1, -1], [0, 1, 2]]
    e = np.exp([0, 0, -1.0])
    assert np.allclose(w[0], e / e.sum(), rtol=1e-15)
    assert w[1].tolist() == [1, 0, 0] and w[2].tolist() == [0, 0, 0] and np.isnan(w[3]).all()


def test_row_gradients_are_difference_quotients():
    # the maps are bilinear: central differences are exact up to rounding
    rng = np.random.default_rng(1)
    T, k, H, R = 4, 3, 5, 14
    dst = rng.permutation(R)[:T * k].reshape(T, k).astype(np.int32)
    dst[2, 1] = -1
    x, rows, w = rng.normal(size=(T, H)), rng.normal(size=(R, H)), rng.normal(size=(T, k))
    gr, gt = rng.normal(size=(R, H)), rng.normal(size=(T, H))
    permute = lambda x, w: float(np.nansum(X.spread(x, dst, w, R) * gr))        # noqa: E731
    combine = lambda r, w: float((X.collect(r, dst, w)[0] * gt).sum())          # noqa: E731
    assert np.abs(X.collect(gr, dst, w)[0] - _diff(lambda v: permute(v, w), x)).max() < 1e-8
    assert np.abs(X.dots(x, gr, dst)[0] - _diff(lambda v: permute(x, v), w)).max() < 1e-8
    d = np.nan_to_num(X.spread(gt, dst, w, R))
    assert np.abs(d - _diff(lambda v: combine(v, w), rows)).max() < 1e-8
    assert np.abs(X.dots(gt, rows, dst)[0] - _diff(lambda v: combine(rows, v), w)).max() < 1e-8


def test_block_rule_by_hand():
    x = np.zeros((1, 144), np.float32)
    x[0, :4] = [448.0, 1.0, 18.0, -17.0]     # scale 1; 17 and 18 around a tie of step 2
    x[0, 128:131] = [7.0, 3.5, 0.0]          # amax 7: scale 1/64, codes of 448, 224, 0
    q, s = X.quantize_rows(x)
    assert s.tolist() == [[1.0, 7.0 / 448.0]]
    assert F.decode_e4m3(q[0, :4]).tolist() == [448.0, 1.0, 18.0, -16.0]
    assert F.decode_e4m3(q[0, 128:131]).tolist() == [448.0, 224.0, 0.0]
    z, sz = X.quantize_rows(np.zeros((1, 16), np.float32))
    assert not z.any() and sz[0, 0] == np.float32(2.0 ** -126)
    v = np.array([[np.inf, 1.0, np.nan, 2.0] + [0.0] * 124 + [np.nan, 4.0] + [0.0] * 14], np.float32)
    q, s = X.quantize_rows(v)
    assert np.isinf(s[0, 0]) and q[0, :4].tolist() == [0x7F, 0, 0x7F, 0]
    assert s[0, 1] == np.float32(4.0 / 448.0) and q[0, 128] == 0x7F


def test_matmul_scales_by_block():
    rng = np.random.default_rng(2)
    a = F.encode_e4m3(rng.normal(size=(5, 160)))
    b = F.encode_e4m3(rng.normal(size=(2, 136, 160)))
    sa, sb = rng.uniform(0.5, 2, (5, 2)), rng.uniform(0.5, 2, (2, 2, 2))
    c = X.matmul(a, b, sa, sb, [0, 2, 2, 5], [1, 0, 0])
    t, n, e = 3, 130, 0
    want = sum(F.decode_e4m3(a[t, k]) * F.decode_e4m3(b[e, n, k]) * sa[t, k // 128] * sb[e, 1, k // 128]
               for k in range(160))
    assert abs(c[t, n] - want) < 1e-9 and np.isfinite(c).all()
