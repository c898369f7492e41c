"""The residual's addition with the root-mean-square norm and its FP8 output on
the GPU against the float64 oracle.

u(dtype) is half a unit in the last place.  h is one fp32 sum, rounded: equal
to the same two steps elsewhere.  The squares' sum of K positive terms runs over
at most 32 terms of a thread, 5 levels of a warp and 16 warps, each 2^-24; the
root halves that; mean, root, reciprocal and the two products add five more:
(53 / 2 + 5) 2^-24, taken as C = 32 2^-24 relative.  Codes in fp32 are exact
steps from v, which the fp32 y shows; else a code is within half a step (2^-4
relative, or 2^-10 of the scale) of v, and v within C.
"""
import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq
from oracle import experts as X
from oracle import formats as F
from oracle import layers as L
from tests._util import DEV, need_gpu, u8
from tests.test_gpu_experts import DTYPES, EPS, TINY, U, close, f64
from tests.test_gpu_guard_regions import Guarded

pytestmark = pytest.mark.gpu
C = 32 * EPS
EPSILON = 1e-6


@pytest.fixture(autouse=True)
def _error_word():
    need_gpu()
    moeq.clear_device_error()
    yield
    assert moeq.get_device_error() == 0


def _rows(n, k, dtype, seed, size=1.0):
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(n, k, device=DEV, generator=g)
    return (x * (size + 20.0 * (torch.rand(n, k, device=DEV, generator=g) < 0.01))).to(dtype)


def _outputs(n, k, dtype, residual, codes, new=None):
    new = new or (lambda s, d: torch.empty(s, dtype=d, device=DEV))
    out = dict(y=new((n, k), dtype), rstd=new((n,), torch.float32))
    if residual:
        out["h"] = new((n, k), dtype)
    if codes:
        out["q"] = new((n, k), torch.uint8)
        out["scales"] = new((n, (k + 127) // 128) if codes == "block" else (n,), torch.float32)
    return out


def _check_codes(out, v, codes):
    """Codes and scales against v float64, itself within C of the kernel's."""
    q, s = F.decode_e4m3(u8(out["q"])), f64(out["scales"])
    n, k = v.shape
    at = np.arange(k) // 128 if codes == "block" else np.zeros(k, np.int64)
    s = s.reshape(n, -1)
    amax = np.zeros_like(s)
    for b in range(s.shape[1]):
        amax[:, b] = np.abs(v[:, at == b]).max(1)
    want = np.maximum(amax / 448.0, 2.0 ** -126)
    assert np.all(np.abs(s - want) <= (C + 2 * EPS) * want)
    err = np.abs(q * s[:, at] - v)
    assert np.all(err <= 2.0 ** -4 * np.abs(v) + 2.0 ** -10 * s[:, at] + (C + 4 * EPS) * np.abs(v))


SHAPES = [(1, 16), (3, 64), (130, 144), (7, 1024), (37, 2048), (5, 2064), (9, 2480), (4, 4096),
          (3, 4112), (6, 7168), (2, 8208), (3, 16384), (305, 272), (1300, 48)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("codes", [None, "block", "row"])
@pytest.mark.parametrize("n,k", SHAPES)
def test_norm_and_gradient(n, k, codes, residual, dtype):
    x, w = _rows(n, k, dtype, n * k), (1 + 0.2 * _rows(1, k, torch.float32, 3)[0]).to(dtype)
    res = _rows(n, k, dtype, 4, 3.0) if residual else None
    out = _outputs(n, k, dtype, residual, codes)
    moeq.add_rms_norm(x, w, residual=res, eps=EPSILON, **out)
    h = (x.float() + res.float()).to(dtype) if residual else x
    if residual:
        assert torch.equal(out["h"], h)
    v, rstd = L.rms_norm(f64(h), f64(w), EPSILON)
    close(out["rstd"], rstd, C * rstd)
    close(out["y"], v, (C + U[dtype]) * np.abs(v) + TINY[dtype])
    if codes and dtype == torch.float32:                   # y is v: the codes to the bit
        y = out["y"].cpu().numpy()
        if codes == "block":
            q, s = X.quantize_rows(y)
        else:
            q, s = (np.stack(a) for a in zip(*(X._codes(r, np.abs(r).max()) for r in y)))
        assert np.array_equal(u8(out["q"]), q) and np.array_equal(out["scales"].cpu().numpy(), s)
    elif codes:
        _check_codes(out, v, codes)
    if codes == "row":
        return
    dy = _rows(n, k, dtype, 5)
    dh = _rows(n, k, dtype, 6) if residual else None
    dx, dw = torch.empty_like(dy), torch.empty(k, device=DEV)
    moeq.add_rms_norm_grad(dy, h, w, out["rstd"], dx, d_weight=dw, d_h=dh)
    ref, ref_dw, mag = L.rms_norm_grad(f64(h), f64(w), EPSILON, f64(dy), None if dh is None else f64(dh))
    # g and h u^2 mean(g h) by their magnitudes, with the mean's K terms summed as the squares
    g = np.abs(f64(dy) * f64(w))
    size = (g + np.abs(f64(h)) * rstd[:, None] ** 2 * (g * np.abs(f64(h))).mean(1, keepdims=True)) * rstd[:, None]
    tol = 3 * C * size + U[dtype] * np.abs(ref) + TINY[dtype] + (0 if dh is None else EPS * np.abs(f64(dh)))
    close(dx, ref, tol)
    # a thread adds n / 300 rows, a column's parts 38 and 5 more
    close(dw, ref_dw, (C + (n / 300 + 50) * EPS) * mag + 1e-30)


def test_gradient_against_differences():
    rng = np.random.default_rng(1)
    n, k, eps = 3, 24, 1e-2
    h, dy = rng.normal(size=(n, k)).astype(np.float32), rng.normal(size=(n, k)).astype(np.float32)
    w = rng.normal(size=k).astype(np.float32)
    to = lambda a: torch.from_numpy(a).to(DEV)                                       # noqa: E731
    y, rstd, dx, dw = (torch.empty(s, device=DEV) for s in ((n, k), (n,), (n, k), (k,)))
    moeq.add_rms_norm(to(h), to(w), y=y, rstd=rstd, eps=eps)
    moeq.add_rms_norm_grad(to(dy), to(h), to(w), rstd, dx, d_weight=dw)
    loss = lambda a, b: (L.rms_norm(a, b, eps)[0] * dy)                              # noqa: E731
    for j in range(k):
        step = np.zeros((n, k))
        step[:, j] = 1e-4
        diff = (loss(h + step, w).sum(1) - loss(h - step, w).sum(1)) / 2e-4
        assert np.all(np.abs(f64(dx)[:, j] - diff) < 1e-5)      # h^2 / 6 of third derivatives, fp32
        diff = (loss(h, w + step[0]).sum() - loss(h, w - step[0]).sum()) / 2e-4
        assert abs(f64(dw)[j] - diff) < 1e-5


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place_and_strided(dtype):
    n, k = 33, 2480
    big, bigr = _rows(n, k + 64, dtype, 1), _rows(n, k + 8, dtype, 2)
    w = _rows(1, k, dtype, 3)[0]
    want = _outputs(n, k, dtype, True, "block")
    moeq.add_rms_norm(big[:, :k].contiguous(), w, residual=bigr[:, :k].contiguous(), **want)
    got = _outputs(n, k, dtype, True, "block")
    moeq.add_rms_norm(big[:, :k], w, residual=bigr[:, :k], **got)
    assert all(torch.equal(want[f], got[f]) for f in want)
    # the stream in place, y over x
    x, r = big[:, :k].contiguous(), bigr[:, :k].contiguous()
    got = dict(got, h=r, y=x)
    moeq.add_rms_norm(x, w, residual=r, **got)
    assert all(torch.equal(want[f], got[f]) for f in want)
    # the gradient over each of its inputs
    dy, dh, dx = _rows(n, k, dtype, 4), _rows(n, k, dtype, 5), torch.empty(n, k, dtype=dtype, device=DEV)
    dw, dw2 = torch.empty(k, device=DEV), torch.empty(k, device=DEV)
    moeq.add_rms_norm_grad(dy, want["h"], w, want["rstd"], dx, d_weight=dw, d_h=dh)
    for over in range(3):
        a = [dy.clone(), want["h"].clone(), dh.clone()]
        moeq.add_rms_norm_grad(a[0], a[1], w, want["rstd"], a[over], d_weight=dw2, d_h=a[2])
        assert torch.equal(a[over], dx) and torch.equal(dw, dw2)
    moeq.add_rms_norm_grad(dy, want["h"], w, want["rstd"], dx2 := torch.empty_like(dx), d_h=dh)
    assert torch.equal(dx, dx2)                            # without the weight's gradient
    # single outputs are those of all together
    for f in ("y", "q"):
        one = {f: torch.empty_like(want[f])}
        if f == "q":
            one["scales"] = torch.empty_like(want["scales"])
        moeq.add_rms_norm(want["h"], w, **one)
        assert all(torch.equal(one[g], want[g]) for g in one)


def test_special_values():
    inf, nan = float("inf"), float("nan")
    k = 256
    x = torch.ones(6, k, device=DEV)
    x[0] = 0.0
    x[1, 5], x[2, 7], x[3, 200] = nan, inf, -inf
    x[4] = torch.finfo(torch.float32).max
    x[5, :128] = 0.0
    w = torch.ones(k, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        xd, wd = x.to(dtype), w.to(dtype)
        out = _outputs(6, k, dtype, False, "block")
        moeq.add_rms_norm(xd, wd, eps=EPSILON, **out)
        h = xd.float()
        ref = h * (1.0 / (h.square().mean(1, keepdim=True) + EPSILON).sqrt())
        got, s = out["y"].float(), out["scales"]
        assert torch.equal(got.isnan(), ref.to(dtype).isnan()) and not got[0].any()
        fine = ~ref.isnan()
        assert torch.allclose(got[fine], ref[fine], rtol=2 * U[dtype] + C, atol=0)
        assert torch.equal(s[0], torch.full_like(s[0], 2.0 ** -126)) and not out["q"][0].any()
        assert float(s[5, 0]) == 2.0 ** -126
        nans = (u8(out["q"]) & 0x7F) == 0x7F
        assert np.array_equal(nans, got.isnan().cpu().numpy())
    # rows of zeros without an epsilon: 0 * inf
    y = torch.zeros(1, k, device=DEV)
    moeq.add_rms_norm(x[:1], w, y=y, eps=0.0)
    assert y.isnan().all()


def test_no_rows():
    x, w = torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV)
    u, dw = torch.empty(0, device=DEV), torch.full((64,), 7.0, device=DEV)
    moeq.add_rms_norm(x, w, y=torch.empty_like(x), rstd=u)
    moeq.add_rms_norm_grad(x, x, w, u, torch.empty_like(x), d_weight=dw)
    assert not dw.any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,k", [(1, 16), (5, 48), (131, 272), (33, 2064), (7, 4112), (3, 8208), (2, 16384)])
def test_stays_in_its_buffers(n, k, dtype):
    g = Guarded()
    x, w = _rows(n, k, dtype, 1), _rows(1, k, dtype, 2)[0]
    for codes in ("block", "row"):
        out = _outputs(n, k, dtype, True, codes, g)
        moeq.add_rms_norm(x, w, residual=x, **out)
        ws = g((moeq.add_rms_norm_grad_workspace(n, k),), torch.uint8)
        moeq.add_rms_norm_grad(x, out["h"], w, out["rstd"], g((n, k), dtype), d_h=x,
                               d_weight=g((k,), torch.float32), workspace=ws)
    g.check()


def test_offsets_past_32_bits():
    n, k = (1 << 32) // 8192 + 300, 8192 + 16              # bf16: 8.6 GB each
    x = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    x[:] = _rows(64, k, torch.bfloat16, 1).repeat((n + 63) // 64, 1)[:n]
    w = _rows(1, k, torch.bfloat16, 2)[0]
    out = _outputs(n, k, torch.bfloat16, False, "block")
    moeq.add_rms_norm(x, w, **out)
    few = _outputs(64, k, torch.bfloat16, False, "block")
    moeq.add_rms_norm(x[:64], w, **few)
    at = torch.arange(n, device=DEV) % 64
    for f in out:
        for a in range(0, n, 1 << 17):
            assert torch.equal(out[f][a:a + (1 << 17)], few[f][at[a:a + (1 << 17)]])
    dx = torch.empty_like(x)
    del out["q"], out["scales"]
    moeq.add_rms_norm_grad(out["y"], x, w, out["rstd"], dx, d_h=x)
    fx = torch.empty(64, k, dtype=torch.bfloat16, device=DEV)
    moeq.add_rms_norm_grad(few["y"], x[:64], w, few["rstd"], fx, d_h=x[:64])
    for a in range(0, n, 1 << 17):
        assert torch.equal(dx[a:a + (1 << 17)], fx[at[a:a + (1 << 17)]])


def test_streams_and_graphs():
    """Calls on a given stream wait for nothing else; two graphs with workspaces of
    their own replay at the same time with the direct calls' results."""
    n, k = 4000, 2048
    w = _rows(1, k, torch.bfloat16, 3)[0]
    work, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for i, s in enumerate(streams):
        x = _rows(n, k, torch.bfloat16, 10 + i)
        st = dict(x=x, dx=torch.empty_like(x), dw=torch.empty(k, device=DEV),
                  ws=torch.empty(moeq.add_rms_norm_grad_workspace(n, k), dtype=torch.uint8, device=DEV),
                  out=_outputs(n, k, torch.bfloat16, True, "block"))
        work.append(st)

        def step(st, stream=None):
            moeq.add_rms_norm(st["x"], w, residual=st["x"], stream=stream, **st["out"])
            moeq.add_rms_norm_grad(st["x"], st["out"]["h"], w, st["out"]["rstd"], st["dx"],
                                   d_weight=st["dw"], workspace=st["ws"], stream=stream)
        step(st)
        torch.cuda.synchronize()
        st["want"] = [t.clone() for t in (st["dx"], st["dw"], *st["out"].values())]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(st)
        graphs.append(g)
        for t in (st["dx"], st["dw"], *st["out"].values()):
            t.zero_()
        step(st, stream=s)                                  # by its handle
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(st["want"], (st["dx"], st["dw"], *st["out"].values())))
    torch.cuda.synchronize()
    for st in work:
        for t in (st["dx"], st["dw"], *st["out"].values()):
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for st in work:
        assert all(torch.equal(a, b) for a, b in zip(st["want"], (st["dx"], st["dw"], *st["out"].values())))


def test_refusals():
    x, w = torch.zeros(4, 64, device=DEV), torch.zeros(64, device=DEV)
    y, u = torch.zeros(4, 64, device=DEV), torch.zeros(4, device=DEV)
    for kw in (dict(y=y[:3]), dict(y=y.bfloat16()), dict(y=y, residual=x[:, :32]), dict(y=y, rstd=u[:3]),
               dict(q=y), dict(y=y.cpu())):
        with pytest.raises((ValueError, TypeError)):
            moeq.add_rms_norm(x, w, **kw)
    for kw in (dict(), dict(y=y, residual=x), dict(y=y, h=y), dict(q=y.to(torch.uint8)), dict(y=y, eps=-1.0)):
        with pytest.raises(moeq.MoeqError):
            moeq.add_rms_norm(x, w, **kw)
    with pytest.raises(ValueError):
        moeq.add_rms_norm_grad(x, x, w, u, y, d_weight=w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        moeq.add_rms_norm_grad(x, x, w, u, y, d_weight=w, stream=torch.cuda.Stream())
    with pytest.raises(ValueError):
        moeq.add_rms_norm_grad(x, x[:3], w, u, y)
