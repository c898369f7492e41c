"""The router, tokens to rows and back, the FP8 128-block quantizer and the
FP8 block GEMM on the GPU against the float64 oracle (the quantizer, whose
definition is fp32 steps, byte for byte).

Tolerances, all derived from the arithmetic.  u(dtype) is half a unit in the
last place: 2^-8 bf16, 2^-11 fp16 (plus half its subnormal step, 2^-25),
2^-24 fp32.
* router weights: exp(d) is within 2 + 1.173 |d| ulp of 2^-23, its argument
  d = x - m within |d| 2^-24 (absolute, so relative in the result), the sums of
  E positive terms within (E / 32 + 6) 2^-24, the division and the scale 2^-23;
* products and sums of rows: u times the result plus (k + 1) 2^-24 times the
  sum of magnitudes; dot products of H terms: (H + 8) 2^-24 times the sum of
  magnitudes in any order;
* GEMM: max(2 bf16 ulp, 1e-3 rms), as for the other grouped GEMMs.
"""
import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq, synth
from oracle import experts as X
from tests._util import (DEV, assert_gemm_close, bf16_bits, groups_from_counts, need_gpu,
                         to_dev_i32, to_dev_u32, u8)

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
EPS = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, tol):
    got = f64(got)
    assert got.shape == want.shape and np.all(np.isfinite(got) == np.isfinite(want))
    bad = np.abs(got - want) > tol
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want)[bad].max()))


@pytest.fixture(autouse=True)
def _error_word():
    need_gpu()
    moeq.clear_device_error()
    yield


# ------------------------------------------------------------------ router

def _gate(x, k, normalize, scale):
    ids = torch.full((x.shape[0], k), -9, dtype=torch.int32, device=DEV)
    w = torch.full((x.shape[0], k), -9.0, device=DEV)
    moeq.gate_topk(x, ids, w, normalize=normalize, scale=scale)
    return ids, w


def _gate_tol(x, scale):
    spread = np.nan_to_num(x, neginf=0).max(1) - np.where(np.isfinite(x), x, np.inf).min(1)
    spread = np.minimum(np.abs(np.nan_to_num(spread)), 104.0)
    return (2.0 ** -21 + 3.5 * spread * EPS + (x.shape[1] / 32 + 10) * EPS)[:, None] * scale


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (129, 8, 2), (33, 33, 7), (64, 128, 8),
                                   (31, 200, 6), (17, 256, 8), (9, 513, 32), (5, 1024, 10)])
def test_gate_and_gradient(T, E, k, dtype, normalize):
    g = np.random.default_rng(T * E + k)
    x = torch.from_numpy(g.normal(size=(T, E)) * 2).to(dtype)     # bf16 rows hold ties
    if E > 2 * k:
        x[::3, : E // 2] = float("-inf")
    scale = 2.5 if normalize else 1.0
    ids, w = _gate(x.to(DEV), k, normalize, scale)
    ref_ids, ref_w = X.gate_topk(f64(x), k, normalize, scale)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    rel = _gate_tol(f64(x), 1.0)
    close(w, ref_w, rel * ref_w + 1e-37)
    dw = torch.from_numpy(g.normal(size=(T, k))).float()
    dx = torch.full((T, E), 9.0, dtype=dtype, device=DEV)
    moeq.gate_topk_grad(x.to(DEV), ids, dw.to(DEV), dx, normalize=normalize, scale=scale)
    ref = X.gate_topk_grad(f64(x), ref_ids, f64(dw), normalize, scale)
    # every term is a product of weights and d_w's, each within rel; three of them meet
    size = np.abs(f64(dw)).max(1, keepdims=True) * scale
    close(dx, ref, 4 * (rel + 8 * EPS) * size + U[dtype] * np.abs(ref) + TINY[dtype])
    assert moeq.get_device_error() == 0


def test_gate_rows_without_choices():
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[-inf] * 40, [-inf] * 39 + [1.0], [nan] + [0.0] * 39, [nan] * 40,
                      [inf] + [0.0] * 39, [-0.0, 0.0] * 20,
                      [torch.finfo(torch.float32).min] * 40])
    for normalize in (False, True):
        ids, w = _gate(x.to(DEV), 3, normalize, 1.0)
        want_ids, want_w = X.gate_topk(f64(x), 3, normalize, 1.0)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert np.allclose(f64(w), want_w, rtol=1e-6, atol=0, equal_nan=True)
        dx = torch.full_like(x, 7.0, device=DEV)
        moeq.gate_topk_grad(x.to(DEV), ids, torch.ones(7, 3, device=DEV), dx, normalize=normalize)
        assert not dx[:2].any()      # no choice, or a single one: nothing to learn
        assert torch.isfinite(dx[5:]).all()
    assert moeq.get_device_error() == 0


@pytest.mark.parametrize("E,k", [(8, 3), (100, 8), (256, 8), (300, 32), (1024, 9)])
def test_gate_orders_logits_that_differ_in_their_last_bits(E, k):
    """fp32 logits one ulp apart, equal ones and both zeros among them."""
    rng = np.random.default_rng(E)
    base = rng.normal(size=(64, E)).astype(np.float32)
    base[8:16] = 1.0
    base[16:24] = 0.0
    base[24:32] = -3.5
    steps = rng.integers(-3, 4, size=(64, E))
    x = (base.view(np.int32) + np.where(base == 0, 0, steps).astype(np.int32)).view(np.float32)
    x[16:24, ::2] = -0.0
    x[:, ::5] = x[:, 1::5][:, :1]
    ids, w = _gate(torch.from_numpy(x).to(DEV), k, True, 1.0)
    want_ids, want_w = X.gate_topk(x, k, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    close(w, want_w, _gate_tol(x.astype(np.float64), 1.0) * want_w)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [5, 17000])
@pytest.mark.parametrize("E", [1, 8, 16, 32])
def test_gate_takes_every_expert(E, T, dtype):
    """top_k = num_experts: as many rounds as there are logits, with NaN and -inf
    among them, in the last place too; equal logits in order."""
    x = np.tile(np.random.default_rng(E).integers(-2, 3, size=(5, E)).astype(np.float32),
                (T // 5, 1))
    x[1::5, -1] = np.nan
    x[2::5, 0] = -np.inf
    x[3::5, -1] = -np.inf
    ids, _ = _gate(torch.from_numpy(x).to(dtype).to(DEV), E, True, 1.0)
    want, _ = X.gate_topk(x[:5].astype(np.float64), E, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), np.tile(want, (T // 5, 1)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("E,k", [(3, 2), (23, 6), (32, 1), (39, 8), (72, 4), (129, 8)])
def test_gate_many_tokens(E, k, normalize, dtype):
    """Many tokens: against the oracle's rule on whole arrays (a stable sort),
    with masked experts, ties, rows without a choice and NaN rows."""
    T = 40037
    g = torch.Generator(device=DEV)
    g.manual_seed(E)
    x = (torch.randn(T, E, generator=g, device=DEV) * 2).to(dtype)
    if E > 2:
        x[5::7, 1] = x[5::7, 0]
    x[::11, : E // 2] = float("-inf")
    x[17] = float("-inf")
    x[40000, E - 1] = float("nan")
    ids, w = _gate(x, k, normalize, 1.5)
    v = torch.where(torch.isnan(x), float("-inf"), x).double()
    top = torch.sort(v, dim=1, descending=True, stable=True)
    val, want = top.values[:, :k], top.indices[:, :k].int()
    want = torch.where(val > float("-inf"), want, -1)
    assert torch.equal(ids, want)
    over = val if normalize else v
    ref = 1.5 * torch.exp(val - torch.logsumexp(over, 1, keepdim=True)).nan_to_num(0.0)
    row = torch.ones(T, dtype=torch.bool, device=DEV)
    row[40000] = False
    assert torch.isnan(w[40000][ids[40000] >= 0]).all()
    rel = _gate_tol(f64(x[row]), 1.0)
    close(w[row], f64(ref[row]), rel * f64(ref[row]) + 1e-37)


def test_gate_strided_rows_and_bad_ids():
    wide = torch.randn(50, 96, generator=torch.Generator().manual_seed(1)).to(DEV)
    ids, w = _gate(wide[:, :64], 4, True, 1.0)
    ids2, w2 = _gate(wide[:, :64].contiguous(), 4, True, 1.0)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    ids[7, 1] = 64
    dx = torch.empty(50, 64, device=DEV)
    moeq.gate_topk_grad(wide[:, :64], ids, torch.ones(50, 4, device=DEV), dx)
    assert moeq.get_device_error() == moeq.DEVERR_BAD_EXPERT and torch.isfinite(dx).all()
    moeq.clear_device_error()


# ------------------------------------------------- tokens, rows, gradients

def _dst(T, k, R, rng, drop=0.15):
    dst = rng.permutation(R)[:T * k].reshape(T, k).astype(np.int32)
    dst[rng.random((T, k)) < drop] = -1
    if T > 2:
        dst[1] = -1                  # a token whose every choice was dropped
    return dst


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,H,k,strided", [(1, 8, 1, False), (5, 16, 3, True), (33, 264, 2, True),
                                           (130, 120, 4, False), (6, 1536, 4, True),
                                           (7, 1032, 8, False), (3, 4104, 5, True),
                                           (70, 64, 11, False), (2, 8192, 32, False)])
def test_rows_and_gradients(T, H, k, strided, weighted, dtype):
    rng = np.random.default_rng(T * H + k)
    R = T * k + 3
    dst = _dst(T, k, R, rng)

    def wide(n):                     # rows of a wider tensor
        return torch.from_numpy(rng.normal(size=(n, H + 16 if strided else H))).to(dtype).to(DEV)[:, :H]

    x, rows, g_rows, g_out = wide(T), wide(R).contiguous(), wide(R).contiguous(), wide(T)
    w = torch.from_numpy(rng.normal(size=(T, k))).float().to(DEV) if weighted else None
    wn, d = (f64(w) if weighted else None), torch.from_numpy(dst).to(DEV)
    u, tiny = U[dtype], TINY[dtype]

    def check_spread(got, ref):
        untouched = np.isnan(ref)
        assert np.all(f64(got)[untouched] == 7.0)
        ref = np.where(untouched, 7.0, ref)
        # without weights a copy: no rounding at all
        close(got, ref, (u + EPS) * np.abs(ref) + tiny if weighted else 0.0 * ref)

    def check_collect(got, pair):
        close(got, pair[0], u * np.abs(pair[0]) + (k + 1) * EPS * 1.01 * pair[1] + tiny)

    def check_dots(got, pair):
        close(got, pair[0], (H + 8) * EPS * pair[1])
        assert not f64(got)[dst < 0].any()

    out = torch.full((R, H), 7.0, dtype=dtype, device=DEV)
    moeq.permute_topk(x, d, out, weights=w)
    check_spread(out, X.spread(f64(x), dst, wn, R))
    dx, dw = torch.full((T, H), 7.0, dtype=dtype, device=DEV), torch.full((T, k), 7.0, device=DEV)
    moeq.permute_topk_grad(g_rows, d, dx, weights=w, tokens=x, d_weights=dw)
    check_collect(dx, X.collect(f64(g_rows), dst, wn))
    check_dots(dw, X.dots(f64(x), f64(g_rows), dst))

    y = torch.full((T, H), 7.0, dtype=dtype, device=DEV)
    moeq.combine_topk(rows, d, y, weights=w)
    check_collect(y, X.collect(f64(rows), dst, wn))
    dr, dw2 = torch.full((R, H), 7.0, dtype=dtype, device=DEV), torch.full((T, k), 7.0, device=DEV)
    moeq.combine_topk_grad(g_out, d, dr, weights=w, rows=rows, d_weights=dw2)
    check_spread(dr, X.spread(f64(g_out), dst, wn, R))
    check_dots(dw2, X.dots(f64(g_out), f64(rows), dst))
    # without the weights' gradient the other output is the same
    dx2, dr2 = torch.empty_like(dx), torch.full_like(dr, 7.0)
    moeq.permute_topk_grad(g_rows, d, dx2, weights=w)
    moeq.combine_topk_grad(g_out, d, dr2, weights=w)
    assert torch.equal(dx, dx2) and torch.equal(dr, dr2)
    assert moeq.get_device_error() == 0


def test_rows_bad_index_skips_and_reports():
    x = torch.ones(4, 64, device=DEV)
    dst = torch.tensor([[0, 9], [-2, 1], [2, -1], [3, 8]], dtype=torch.int32, device=DEV)
    rows = torch.full((8, 64), 7.0, device=DEV)
    moeq.permute_topk(x, dst, rows)
    assert torch.equal(rows[:4], x) and bool((rows[4:] == 7.0).all())
    assert moeq.get_device_error() == moeq.DEVERR_BAD_INDEX
    moeq.clear_device_error()
    y = torch.empty_like(x)
    moeq.combine_topk(rows, dst, y)
    assert torch.equal(y, x) and moeq.get_device_error() == moeq.DEVERR_BAD_INDEX
    moeq.clear_device_error()


def test_rows_copy_bits_and_carry_infinities():
    x = torch.tensor([0x7FC1, 0xFF80, 0x7F80, 0x0001, 0x8000, 0xFFFF, 1, 2], dtype=torch.int32)
    x = x.to(torch.int16).view(torch.bfloat16).view(1, 8).to(DEV)
    dst = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    rows = torch.zeros(2, 8, dtype=torch.bfloat16, device=DEV)
    moeq.permute_topk(x, dst, rows)
    assert torch.equal(rows.view(torch.int16), x.view(torch.int16).expand(2, 8))
    # an infinite row reaches the tokens that chose it, others' NaN does not
    r = torch.zeros(3, 8, dtype=torch.bfloat16, device=DEV)
    r[0], r[2] = float("inf"), float("nan")
    y = torch.empty(2, 8, dtype=torch.bfloat16, device=DEV)
    moeq.combine_topk(r, torch.tensor([[0, 1], [1, -1]], dtype=torch.int32, device=DEV), y)
    assert torch.isinf(y[0]).all() and not y[1].any()


def test_rows_offsets_past_32_bits():
    # 300000 rows of 16 KB: the last ones start past 2^32 bytes
    T, H = 5, 8192
    R = 300000
    rows = torch.empty(R, H, dtype=torch.bfloat16, device=DEV)
    dst = torch.tensor([[0, R - 1 - t] for t in range(T)], dtype=torch.int32, device=DEV)
    dst[:, 0] += torch.arange(T, dtype=torch.int32, device=DEV)
    x = synth.bf16_normal((T, H), seed=1, device=DEV)
    moeq.permute_topk(x, dst, rows)
    for t in range(T):
        assert torch.equal(rows[R - 1 - t], x[t]) and torch.equal(rows[t], x[t])
    y = torch.empty_like(x)
    moeq.combine_topk(rows, dst, y, weights=torch.full((T, 2), 0.5, device=DEV))
    assert torch.equal(y, x)


# ----------------------------------------------------- FP8 with 128-blocks

def _activations(R, K, seed):
    x = synth.bf16_normal((R, K), 1.0, seed=seed, outlier_p=0.01, outlier_scale=30.0)
    x[0, : min(K, 128)] = 0                                   # a block of zeros
    if R > 2:
        x[2] *= 2.0 ** -100                                   # scales far from 1
        x[1, ::7] = 2.0 ** -133                               # subnormal inputs
        x[1, 1::7] = 0
    return x


def _check_bytes(q, s, ref):
    got, want = u8(q), ref[0]
    nan = (want & 0x7F) == 0x7F
    assert np.array_equal(got[~nan], want[~nan]) and np.all(got[nan] & 0x7F == 0x7F)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), ref[1].view(np.uint32))


@pytest.mark.parametrize("R,K,pad", [(1, 16, 0), (300, 592, 0), (64, 1376, 0), (7, 512, 24), (3, 128, 8), (5, 144, 0), (17, 272, 16),
                                     (4, 1040, 0), (2, 2064, 0), (130, 384, 0), (3, 7168, 0)])
def test_quantize_rows_bit_exact(R, K, pad):
    wide = _activations(R, K + pad, seed=K + R)
    x = wide.to(DEV)[:, :K]
    q = torch.full((R, K), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((R, (K + 127) // 128), -1.0, device=DEV)
    moeq.quantize_fp8_block(x, q, s)
    _check_bytes(q, s, X.quantize_rows(wide[:, :K].float().numpy()))


@pytest.mark.parametrize("T,K,k", [(1, 128, 1), (9, 400, 3), (33, 1024, 8), (2, 2576, 20)])
def test_quantize_routed_tokens_bit_exact(T, K, k):
    rng = np.random.default_rng(T)
    R = T * k + 2
    dst = _dst(T, k, R, rng)
    x = _activations(T, K, seed=K)
    q = torch.full((R, K), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((R, (K + 127) // 128), -1.0, device=DEV)
    moeq.quantize_fp8_block_topk(x.to(DEV), torch.from_numpy(dst).to(DEV), q, s)
    rq, rs = X.quantize_rows(x.float().numpy())
    want_q, want_s = np.full((R, K), 0xA5, np.uint8), np.full(s.shape, -1.0, np.float32)
    for t, j in np.ndindex(T, k):
        if dst[t, j] >= 0:
            want_q[dst[t, j]], want_s[dst[t, j]] = rq[t], rs[t]
    _check_bytes(q, s, (want_q, want_s))
    assert moeq.get_device_error() == 0
    bad = torch.from_numpy(dst).to(DEV)
    bad[0, 0] = R
    moeq.quantize_fp8_block_topk(x.to(DEV), bad, q, s)
    assert moeq.get_device_error() == moeq.DEVERR_BAD_INDEX
    moeq.clear_device_error()


def test_quantize_rows_special_values():
    x = torch.zeros(4, 256)
    x[0, 3], x[0, 130] = float("inf"), 5.0
    x[1, 0], x[1, 1] = float("nan"), 2.0
    x[2, :128] = float("nan")
    x[3] = torch.finfo(torch.bfloat16).max
    x[3, 9] = -float("inf")
    x = x.bfloat16()
    q = torch.empty((4, 256), dtype=torch.uint8, device=DEV)
    s = torch.empty((4, 2), device=DEV)
    moeq.quantize_fp8_block(x.to(DEV), q, s)
    _check_bytes(q, s, X.quantize_rows(x.float().numpy()))


@pytest.mark.parametrize("R,I", [(1, 16), (9, 384), (3, 592), (7, 144), (130, 128), (33, 1536), (5, 2064)])
def test_swiglu_quantize_bit_exact(R, I):
    y = synth.bf16_normal((R, 2 * I), 2.0, seed=I)
    y[0, 0], y[R - 1, 2] = -float("inf"), 3e38
    q = torch.full((R, I), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((R, (I + 127) // 128), -1.0, device=DEV)
    moeq.swiglu_quantize_fp8_block(y.to(DEV), q, s)
    with np.errstate(all="ignore"):
        ref = X.swiglu_quantize(y.float().numpy())
    _check_bytes(q, s, ref)


def test_swiglu_quantize_large_is_the_small_one():
    """Past 2^25 values the SiLU comes from a table: the bytes of the same rows
    in a small call, every bf16 gate among them."""
    R, I = 32800, 1040
    y = synth.bf16_normal((R, 2 * I), 2.0, seed=3, device=DEV)
    bits = torch.arange(1 << 16, device=DEV, dtype=torch.int32).to(torch.int16)
    y[-64:].view(torch.int16).view(-1, 2)[: 1 << 16, 0] = bits   # 64 rows hold 66560 gates
    q = torch.zeros((R, I), dtype=torch.uint8, device=DEV)
    s = torch.zeros((R, (I + 127) // 128), device=DEV)
    moeq.swiglu_quantize_fp8_block(y, q, s)
    for r0 in range(0, R, 8200):
        q2, s2 = torch.ones_like(q[:8200]), torch.ones_like(s[:8200])
        moeq.swiglu_quantize_fp8_block(y[r0:r0 + 8200], q2, s2)
        assert torch.equal(q[r0:r0 + 8200], q2)
        assert torch.equal(s[r0:r0 + 8200].view(torch.int32), s2.view(torch.int32))


@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (3, 128, 128), (2, 200, 336), (4, 136, 1024)])
def test_quantize_weight_bit_exact(E, N, K):
    w = synth.bf16_normal((E, N, K), 0.1, seed=N, outlier_p=0.001, outlier_scale=100.0)
    w[0, 0, 0] = 0
    q = torch.full((E, N, K), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((E, (N + 127) // 128, (K + 127) // 128), -1.0, device=DEV)
    moeq.quantize_fp8_block_weight(w.to(DEV), q, s)
    _check_bytes(q, s, X.quantize_weight(w.float().numpy()))


# --------------------------------------------------------- FP8 block GEMM

CANARY = -12288.0


def _gemm_inputs(T, E, N, K, seed):
    kb, nb = (K + 127) // 128, (N + 127) // 128
    a = synth.e4m3_normal((T, K), 50.0, seed=seed)
    b = synth.e4m3_normal((E, N, K), 50.0, seed=seed + 1)
    sa = synth.uniform((T, kb), 0.002, 0.02, seed=seed + 2)
    sb = synth.uniform((E, nb, kb), 0.002, 0.02, seed=seed + 3)
    return a, b, sa, sb


def _gemm(a, b, sa, sb, ro, ids, **kw):
    c = torch.full((a.shape[0], b.shape[1]), CANARY, dtype=torch.bfloat16, device=DEV)
    moeq.grouped_matmul_fp8_block(c, a.to(DEV), b.to(DEV), sa.to(DEV), sb.to(DEV), to_dev_u32(ro),
                                  to_dev_i32(ids), **kw)
    return c


@pytest.mark.parametrize("counts,ids,N,K,tail", [
    ([1], [0], 8, 16, 0),
    ([7, 16, 9], [2, 0, 3], 64, 128, 0),
    ([1, 0, 1, 2], [1, 1, 0, 2], 136, 144, 3),
    ([0, 1, 127, 129, 3, 200], [4, 0, 2, 5, 1, 3], 264, 400, 5),
    ([300, 128, 0, 33], [1, 0, 2, 1], 520, 1168, 0),
    ([5, 90], [0, 1], 72, 1024, 1),
    ([260], [0], 384, 528, 0),
    ([40, 2, 8, 8, 8, 1, 1, 64], [0, 1, 2, 3, 4, 5, 6, 7], 1000, 2048, 0),
])
def test_block_gemm_against_oracle(counts, ids, N, K, tail):
    ro, ids = groups_from_counts(counts, ids)
    T, E = int(ro[-1]) + tail, max(ids) + 1
    a, b, sa, sb = _gemm_inputs(T, E, N, K, seed=N + K)
    c = _gemm(a, b, sa, sb, ro, ids, max_tokens_per_expert=max(counts))
    ref = X.matmul(u8(a), u8(b), sa.numpy(), sb.numpy(), ro, ids)
    n = int(ro[-1])
    assert_gemm_close(bf16_bits(c)[:n], ref[:n])
    assert bool((c[n:] == CANARY).all())
    assert torch.equal(c[:n], _gemm(a, b, sa, sb, ro, ids)[:n])   # the hint changes nothing
    assert moeq.get_device_error() == 0


def test_block_gemm_scales_are_exact_powers():
    """Power-of-two scales factor out exactly: rescaling both sides of one K
    block, one row and one column block shifts exponents only."""
    ro, ids = groups_from_counts([150, 30])
    a, b, sa, sb = _gemm_inputs(180, 2, 256, 384, seed=5)
    sa, sb = torch.full_like(sa, 0.5), torch.full_like(sb, 0.25)
    c = _gemm(a, b, sa, sb, ro, ids).float()
    sa[3] *= 4.0
    sb[1, 1] *= 8.0
    want = c.clone()
    want[3] *= 4.0
    want[150:, 128:256] *= 8.0
    got = _gemm(a, b, sa, sb, ro, ids).float()
    assert torch.equal(got, want)
    sa[:, 1] *= 2.0 ** -7
    sb[:, :, 1] *= 2.0 ** 7
    assert torch.equal(_gemm(a, b, sa, sb, ro, ids).float(), want)


def test_block_gemm_keeps_nonfinite_values_in_their_row_and_column():
    ro, ids = groups_from_counts([140, 60])
    a, b, sa, sb = _gemm_inputs(200, 2, 136, 272, seed=9)
    clean = _gemm(a, b, sa, sb, ro, ids)
    ab, bb = a.view(torch.uint8).clone(), b.view(torch.uint8).clone()
    ab[137, 200] = 0x7F
    bb[1, 130, 5] = 0xFF
    sa2 = sa.clone()
    sa2[20, 0] = float("inf")
    got = _gemm(ab.view(torch.float8_e4m3fn), bb.view(torch.float8_e4m3fn), sa2, sb, ro, ids)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[137], bad[140:, 130], bad[20] = True, True, True
    assert not torch.isfinite(got[bad]).any()
    assert torch.equal(got[~bad], clean[~bad])


def test_block_gemm_bad_groups_are_skipped():
    a, b, sa, sb = _gemm_inputs(64, 2, 64, 128, seed=3)
    good = _gemm(a, b, sa, sb, [0, 20, 40, 64], [0, 1, 0])
    c = _gemm(a, b, sa, sb, [0, 20, 40, 64], [0, 2, 0])
    assert moeq.get_device_error() == moeq.DEVERR_BAD_EXPERT
    assert torch.equal(c[:20], good[:20]) and torch.equal(c[40:], good[40:])
    assert bool((c[20:40] == CANARY).all())
    moeq.clear_device_error()
    c = _gemm(a, b, sa, sb, [0, 20, 10, 65], [0, 1, 0])
    assert moeq.get_device_error() == moeq.DEVERR_BAD_OFFSETS
    assert torch.equal(c[:20], good[:20]) and bool((c[20:] == CANARY).all())
    moeq.clear_device_error()


@pytest.mark.parametrize("G", [512, 1024])
def test_block_gemm_many_groups(G):
    counts = np.random.default_rng(G).integers(0, 4, G)
    ro, _ = groups_from_counts(counts)
    ids = np.arange(G, dtype=np.int32) % 5
    a, b, sa, sb = _gemm_inputs(int(ro[-1]), 5, 136, 256, seed=G)
    c = _gemm(a, b, sa, sb, ro, ids)
    assert_gemm_close(bf16_bits(c), X.matmul(u8(a), u8(b), sa.numpy(), sb.numpy(), ro, ids))


def test_block_gemm_decode_shape():
    """The decode workload's K and N on few experts, one to five rows each."""
    ro, ids = groups_from_counts([1, 5, 2, 3], [3, 0, 1, 2])
    a, b, sa, sb = _gemm_inputs(11, 4, 4096, 7168, seed=2)
    c = _gemm(a, b, sa, sb, ro, ids, max_tokens_per_expert=5)
    assert_gemm_close(bf16_bits(c), X.matmul(u8(a), u8(b), sa.numpy(), sb.numpy(), ro, ids))


# ------------------------------------------------------- the layer's calls

def test_calls_run_on_the_given_stream():
    """Every call goes to the stream it is given: inputs are filled on that
    stream only, behind work that keeps it busy."""
    s = torch.cuda.Stream()
    x, g = torch.zeros(64, 256, device=DEV), torch.zeros(64, 8, device=DEV)
    ids, w = torch.empty(64, 2, dtype=torch.int32, device=DEV), torch.empty(64, 2, device=DEV)
    rows, y = torch.zeros(128, 256, device=DEV), torch.zeros(64, 256, device=DEV)
    dst = torch.arange(128, dtype=torch.int32, device=DEV).view(64, 2)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(8):
            big = (big @ big).clamp_(-1, 1)
        x.fill_(3.0)
        g[:, 5] = 1.0
    moeq.gate_topk(g, ids, w, stream=s)
    moeq.permute_topk(x, dst, rows, stream=s)
    moeq.combine_topk(rows, dst, y, weights=w, stream=s)
    s.synchronize()
    assert bool((ids[:, 0] == 5).all()) and bool((rows == 3.0).all())
    assert torch.allclose(y, torch.full_like(y, 3.0), rtol=4 * EPS + 2.0 ** -21)


def test_layer_in_a_cuda_graph_is_the_same():
    """Router, routing, quantizer, both products and the way back, captured in
    a graph and replayed on new tokens: the bytes of the direct calls."""
    T, E, k, H, I = 96, 16, 4, 256, 128
    R = T * k
    wg = synth.bf16_normal((E, 2 * I, H), 0.1, seed=1, device=DEV)
    wd = synth.bf16_normal((E, H, I), 0.1, seed=2, device=DEV)
    f8 = lambda *s: torch.empty(s, dtype=torch.float8_e4m3fn, device=DEV)        # noqa: E731
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)               # noqa: E731
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)             # noqa: E731
    qg, sg = f8(E, 2 * I, H), torch.empty(E, 2, 2, device=DEV)
    qd, sd = f8(E, H, I), torch.empty(E, 2, 1, device=DEV)
    moeq.quantize_fp8_block_weight(wg, qg, sg)
    moeq.quantize_fp8_block_weight(wd, qd, sd)
    x, logits = bf(T, H), torch.empty(T, E, device=DEV)
    ids, w, ro, eids, src, dst = i32(T, k), torch.empty(T, k, device=DEV), i32(E + 1), i32(E), i32(R), i32(T, k)
    qa, sa, qh, sh = f8(R, H), torch.empty(R, 2, device=DEV), f8(R, I), torch.empty(R, 1, device=DEV)
    y, z, out = bf(R, 2 * I), bf(R, H), bf(T, H)

    def layer():
        moeq.gate_topk(logits, ids, w)
        moeq.route_topk(ids, ro, eids, src, dst_info=dst)
        moeq.quantize_fp8_block_topk(x, dst, qa, sa)
        moeq.grouped_matmul_fp8_block(y, qa, qg, sa, sg, ro, eids)
        moeq.swiglu_quantize_fp8_block(y, qh, sh)
        moeq.grouped_matmul_fp8_block(z, qh, qd, sh, sd, ro, eids)
        moeq.combine_topk(z, dst, out, weights=w)

    def fill(seed):
        x.copy_(synth.bf16_normal((T, H), 1.0, seed=seed, device=DEV))
        logits.copy_(synth.uniform((T, E), -3, 3, seed=seed + 50, device=DEV))

    fill(1)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (2, 3):
        fill(seed)
        layer()
        want = out.clone()
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    # the whole layer against plain float64 arithmetic on the quantized weights:
    # activations are rounded to 3 bits twice (2^-4 relative each, random signs)
    deq = lambda q, s: (q.double() * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2))  # noqa: E731
    gu, dn = deq(qg, sg), deq(qd, sd)
    ref = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for j in range(k):
        e = ids[:, j].long()
        v = torch.einsum("th,tnh->tn", x.double(), gu[e])
        h = torch.nn.functional.silu(v[:, 0::2]) * v[:, 1::2]
        ref += w[:, j, None].double() * torch.einsum("ti,thi->th", h, dn[e])
    assert float((out.double() - ref).norm() / ref.norm()) < 2 * 2.0 ** -4
    assert moeq.get_device_error() == 0


def test_block_gemm_refuses_short_group_tables():
    a = torch.zeros(4, 128, dtype=torch.uint8, device=DEV)
    b = torch.zeros(2, 8, 128, dtype=torch.uint8, device=DEV)
    c = torch.zeros(4, 8, dtype=torch.bfloat16, device=DEV)
    sa, sb = torch.ones(4, 1, device=DEV), torch.ones(2, 1, 1, device=DEV)
    offsets = torch.zeros(3, dtype=torch.int32, device=DEV)
    ids = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="too short"):
        moeq.grouped_matmul_fp8_block(c, a, b, sa, sb, offsets[:2], ids)
    with pytest.raises(ValueError, match="too short"):
        moeq.grouped_matmul_fp8_block(c, a, b, sa, sb, offsets, ids, num_active_experts=3)
    moeq.grouped_matmul_fp8_block(c, a, b, sa, sb, offsets, ids)
    assert moeq.get_device_error() == 0
