"""The epilogue's activations and their gradient over all of bf16's range, on the GPU
against the float64 oracle; tolerances as in test_gpu_epilogue."""
import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq
from oracle import formats as F
from oracle import layers as L
from tests._util import DEV, need_gpu, to_dev_i32, to_dev_u32, u8
from tests.test_gpu_epilogue import ACTS, BF16
from tests.test_gpu_experts import EPS, U, close, f64

pytestmark = pytest.mark.gpu
MAX = float(torch.finfo(BF16).max)


@pytest.fixture(autouse=True)
def _error_word():
    need_gpu()
    moeq.clear_device_error()
    yield
    assert moeq.get_device_error() == 0


def _values(dtype=BF16):
    size = [0.0, 1e-40, 1e-30, 0.5, 3.0, 9.0, 11.0, 16.0, 60.0, 87.0, 88.5, 104.0, 1e5, 1e9, 1e12, 1.2e13, 2e13, 1e18, 1.8e19,
            2e19, 1e20, 1e26, 1e32, 1e38, MAX]
    v = torch.tensor(size + [-s for s in size], dtype=torch.float64)
    return torch.cat([v, v.new_zeros(-len(v) % 16)]).to(dtype)


def _grad(dc, z, act, **kw):
    T, N = dc.shape
    q, s = torch.zeros(T, N, dtype=torch.uint8, device=DEV), torch.zeros(T, (N + 127) // 128, device=DEV)
    dz, db = torch.zeros(T, N, dtype=BF16, device=DEV), torch.zeros(1, N, device=DEV)
    moeq.grouped_epilogue_grad(dc, to_dev_u32([0, T]), to_dev_i32([0]), 1, z=z if act else None, activation=act, q=q,
                               scales=s, d_z=dz, d_bias=db)
    return q, s, dz, db


@pytest.mark.parametrize("act", ACTS)
def test_slopes_of_every_size(act):
    """Each value in each column's rows, so that one that is wrong is in the bias's sum."""
    v = _values()
    T, N = 9, len(v)
    z = torch.stack([v.roll(r) for r in range(T)]).to(DEV)
    dc = torch.linspace(-2, 2, T * N).view(T, N).to(BF16).to(DEV)
    q, s, dz, db = _grad(dc, z, act)
    ref, ref_db, mag = L.epilogue_grad(f64(dc), f64(z) if act else None, act, np.zeros(T, int), 1)
    assert np.isfinite(ref).all()
    err = 1.5e-6 * np.abs(f64(dc)) + 2 * EPS * np.abs(ref)
    close(dz, ref, err + U[BF16] * np.abs(ref))
    close(db, ref_db, err.sum(0)[None] + 12 * EPS * mag + 1e-30)
    sv = f64(s)
    assert np.all(np.abs(sv[:, 0] - np.abs(ref).max(1) / 448) <= err.max(1) / 448 + 2 * EPS * sv[:, 0])
    off = np.abs(F.decode_e4m3(u8(q)) * sv - ref)
    assert np.all(off <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * sv + 1.1 * err)


@pytest.mark.parametrize("rows", [3, 4000])
@pytest.mark.parametrize("act", ACTS)
def test_activations_of_every_size(act, rows):
    """A product of zeros: z is the bias, c its activation, in each of the product's forms."""
    b = _values(torch.float32)
    N, K = len(b), 128
    zero = torch.zeros(rows, K, dtype=torch.uint8, device=DEV)
    w = torch.zeros(1, N, K, dtype=torch.uint8, device=DEV)
    one = torch.ones(rows, 1, device=DEV)
    ws = torch.ones(1, (N + 127) // 128, 1, device=DEV)
    off, ids = to_dev_u32([0, rows]), to_dev_i32([0])
    zv = f64(b)
    want = np.tile(L.activate(zv, act)[0], (rows, 1))
    # sigma and Phi within 1.5e-6 of 1, c a product with z; where they are small, 1.5e-6 of z and
    # z past what is not 0 in fp32 by then
    tol = U[BF16] * np.abs(want) + 1.5e-6 * np.where(np.abs(zv) < 110, np.abs(zv), np.abs(want)) + 2.0 ** -126
    for res in (None, torch.zeros(rows, N, dtype=BF16, device=DEV)):
        for saved in (False, True):
            c = torch.full((rows, N), 7.0, dtype=BF16, device=DEV)
            z = torch.full_like(c, 7.0) if saved else None
            moeq.grouped_matmul_fp8_block_epilogue(c, zero, w, one, ws, off, ids, bias=b.view(1, N).to(DEV),
                                                   activation=act, residual=res, z=z)
            close(c, want, tol)
            if saved:
                assert torch.equal(z, b.to(BF16).to(DEV).expand(rows, N))


@pytest.mark.parametrize("act", ACTS)
def test_gradient_of_nan_and_infinities(act):
    """A NaN z makes the slope NaN whatever the activation, as it does the activation; an
    infinite one where the formula has infinity times 0 (all but relu).  A NaN or infinite
    d_c stays in its element, its column's sum and, as a code, in its element."""
    inf, nan = float("inf"), float("nan")
    T, N = 6, 144
    z = torch.randn(T, N, generator=torch.Generator().manual_seed(1)).to(BF16)
    dc = torch.randn(T, N, generator=torch.Generator().manual_seed(2)).to(BF16)
    z[0, 3], z[1, 20], z[2, 37], z[3, 130] = nan, inf, -inf, nan
    dc[4, 50], dc[4, 60], dc[5, 140] = nan, inf, -inf
    z[4, 50], z[4, 60], z[5, 140] = 1.0, 2.0, 0.5
    q, s, dz, db = _grad(dc.to(DEV), z.to(DEV), act)
    with np.errstate(invalid="ignore"):
        ref, ref_db, _ = L.epilogue_grad(f64(dc), f64(z) if act else None, act, np.zeros(T, int), 1)
    got, sums = f64(dz), f64(db)
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isinf(got), np.isinf(ref))
    assert np.array_equal(np.isnan(sums), np.isnan(ref_db)) and np.array_equal(np.isinf(sums), np.isinf(ref_db))
    if act:
        assert np.isnan(got[0, 3]) and np.isnan(got[3, 130])
    fine = np.isfinite(ref)
    tol = 1.6e-6 * np.abs(f64(dc)[fine]) + (U[BF16] + 2 * EPS) * np.abs(ref[fine])
    assert np.all(np.abs(got[fine] - ref[fine]) <= tol)
    assert np.array_equal(np.isnan(F.decode_e4m3(u8(q))), ~fine)   # an infinity's code is NaN
