"""The FP8 block product with bias, activation and residual, and its epilogue's
gradient, on the GPU against the float64 oracle.

Product: z as for the product without epilogue, within max(2 bf16 ulp, 1e-3
rms); an activation's slope is at most 1.13, so c is within max(2 bf16 ulp, 1.2e-3
rms of z) of its definition.  Gradient: with p = sigma(u) and 1 - p within (4 + 1.2
|u|) 2^-23 relative and z u' at most 3 |u|, the slope p (1 + z u' (1 - p)) is within
1.5e-6; gelu's within 7.5e-8 (the formula's bound for Phi) and as much for z phi(z).
A bias's gradient sums rows in fp32, 2^-24 of the magnitudes for each level of the
order: 16 rows of a thread, 8 warps, then the tiles.
"""
import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq, synth
from oracle import experts as X
from oracle import formats as F
from oracle import layers as L
from tests._util import (DEV, assert_gemm_close, bf16_bits, groups_from_counts, need_gpu,
                         to_dev_i32, to_dev_u32, u8)
from tests.test_gpu_experts import EPS, U, _gemm_inputs, close, f64
from tests.test_gpu_guard_regions import Guarded

pytestmark = pytest.mark.gpu
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _error_word():
    need_gpu()
    moeq.clear_device_error()
    yield
    assert moeq.get_device_error() == 0


# ---------------------------------------------------------------- forward

def _case(counts, ids, N, K, tail, seed=1):
    ro, ids = groups_from_counts(counts, ids)
    T, E = int(ro[-1]) + tail, int(max(ids)) + 1
    a, b, sa, sb = _gemm_inputs(T, E, N, K, seed=seed)
    return ro, ids, T, E, (a, b, sa, sb)


def _scaled(ins, rms):
    """The operands with scales that make z's rms about that."""
    a, b, sa, sb = ins
    K = a.shape[1]
    va, vb = F.decode_e4m3(u8(a)), F.decode_e4m3(u8(b))
    at = np.arange(K) // 128
    size = (np.sqrt(np.mean((va * f64(sa)[:, at]) ** 2)) * np.sqrt(K)
            * np.sqrt(np.mean((vb * f64(sb).repeat(128, 1)[:, :b.shape[1]][:, :, at]) ** 2)))
    return a, b, sa * (rms / size), sb


@pytest.mark.parametrize("counts,ids,N,K,tail", [
    ([1], [0], 8, 16, 0), ([0, 3, 0, 70], [1, 0, 1, 2], 264, 400, 3), ([33], [0], 1000, 2720, 0),
    ([64, 1, 63], [2, 0, 1], 128, 128, 5), ([300, 0, 129, 2000], [3, 1, 0, 2], 520, 1040, 7),
    ([128] * 32 + [4], None, 264, 272, 0)])
@pytest.mark.parametrize("act", ACTS)
def test_product_against_oracle(counts, ids, N, K, tail, act):
    ro, ids, T, E, ins = _case(counts, ids, N, K, tail)
    a, b, sa, sb = (t.to(DEV) for t in _scaled(ins, 1.5))
    bias = torch.randn(E, N, device=DEV, generator=torch.Generator(DEV).manual_seed(2))
    res = synth.bf16_normal((T, N), 2.0, seed=3, device=DEV)
    off, eid = to_dev_u32(ro), to_dev_i32(ids)
    experts = L.row_experts(ro, ids, T)
    rows = experts >= 0
    ref = X.matmul(u8(a), u8(b), f64(sa), f64(sb), ro, ids)[rows]
    for use_bias in (False, True):
        for use_res in (False, True):
            c, z = (torch.full((T, N), 7.0, dtype=BF16, device=DEV) for _ in range(2))
            moeq.grouped_matmul_fp8_block_epilogue(
                c, a, b, sa, sb, off, eid, bias=bias if use_bias else None, activation=act,
                residual=res if use_res else None, z=z)
            zr = ref + (f64(bias)[experts[rows]] if use_bias else 0.0)
            assert_gemm_close(bf16_bits(z)[rows], zr)
            want = L.epilogue(zr, act, f64(res)[rows] if use_res else None)
            ulp = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 1e-300))) - 7)
            tol = np.maximum(2 * ulp, 1.2e-3 * np.sqrt(np.mean(zr ** 2)))
            got = f64(c)
            assert np.all(np.abs(got[rows] - want) <= tol)
            assert (got[~rows] == 7).all() and (f64(z)[~rows] == 7).all()
            # without saving z, and with the residual's own buffer as output
            again = res.clone() if use_res else torch.full_like(c, 7.0)
            moeq.grouped_matmul_fp8_block_epilogue(
                again, a, b, sa, sb, off, eid, bias=bias if use_bias else None, activation=act,
                residual=again if use_res else None)
            assert torch.equal(again[rows], c[rows])


def _plain(ins, ro, ids, T, N):
    c = torch.zeros(T, N, dtype=BF16, device=DEV)
    a, b, sa, sb = ins
    moeq.grouped_matmul_fp8_block(c, a, b, sa, sb, to_dev_u32(ro), to_dev_i32(ids))
    return c


@pytest.mark.parametrize("counts,N,K", [([5, 90], 136, 400), ([1, 0, 17], 1000, 2720),
                                        ([2000, 3000], 520, 1040)])
def test_epilogue_is_that_of_the_plain_product(counts, N, K):
    """Saved z without bias is the plain product's bits; c its activation."""
    ro, ids, T, E, ins = _case(counts, None, N, K, 0)
    ins = [t.to(DEV) for t in _scaled(ins, 1.0)]
    a, b, sa, sb = ins
    plain = _plain(ins, ro, ids, T, N)
    c, z = torch.zeros_like(plain), torch.zeros_like(plain)
    off, eid = to_dev_u32(ro), to_dev_i32(ids)
    moeq.grouped_matmul_fp8_block_epilogue(c, a, b, sa, sb, off, eid, activation="relu", z=z)
    assert torch.equal(z, plain) and torch.equal(c, plain.clamp_min(0))
    moeq.grouped_matmul_fp8_block_epilogue(c, a, b, sa, sb, off, eid, bias=torch.zeros(E, N, device=DEV))
    assert torch.equal(c, plain)
    moeq.grouped_matmul_fp8_block_epilogue(c, a, b, sa, sb, off, eid)
    assert torch.equal(c, plain)
    res = torch.zeros_like(plain)
    moeq.grouped_matmul_fp8_block_epilogue(c, a, b, sa, sb, off, eid, residual=res)
    assert torch.equal(c, plain)


@pytest.mark.parametrize("K", [16, 128, 144, 256, 384, 400, 512, 528, 1008, 1168, 2176])
@pytest.mark.parametrize("counts,N", [([1], 8), ([64, 65], 72), ([3, 0, 130], 200), ([64], 9728), ([64], 9736),
                                      ([70] * 20, 384)])
def test_every_tail_of_a_reduction_and_the_border_of_the_tiles(counts, N, K):
    ro, ids, T, E, ins = _case(counts, None, N, K, 0)
    ins = [t.to(DEV) for t in _scaled(ins, 1.0)]
    a, b, sa, sb = ins
    plain = _plain(ins, ro, ids, T, N)
    res = synth.bf16_normal((T, N), 1.0, seed=5, device=DEV)
    c, z = torch.full_like(plain, 7.0), torch.full_like(plain, 7.0)
    moeq.grouped_matmul_fp8_block_epilogue(c, a, b, sa, sb, to_dev_u32(ro), to_dev_i32(ids), z=z, activation="relu",
                                           residual=res)
    assert torch.equal(z, plain)
    # want takes the product rounded to bf16, at most U |product| off, U |plain| (1 + 2 U);
    # c is the exact product's sum rounded: U |that sum|, itself within the first of want;
    # 1e-6 for the sum and the product in fp32
    first = U[BF16] * (1 + 2 * U[BF16]) * np.abs(f64(plain))
    want = f64(plain).clip(0) + f64(res)
    tol = first + U[BF16] * (np.abs(want) + first) + 1e-6 * (np.abs(f64(plain)) + np.abs(f64(res)))
    assert np.all(np.abs(f64(c) - want) <= tol)


def test_nonfinite_values_stay_in_their_elements():
    inf, nan = float("inf"), float("nan")
    ro, ids, T, E, ins = _case([40, 30], None, 264, 256, 0)
    a, b, sa, sb = (t.to(DEV) for t in _scaled(ins, 1.0))
    bias = torch.zeros(E, 264, device=DEV)
    bias[0, 5], bias[1, 7] = nan, inf
    res = torch.zeros(T, 264, dtype=BF16, device=DEV)
    res[3, 200], res[50, 100] = -inf, nan
    for act in ACTS:
        c = torch.zeros(T, 264, dtype=BF16, device=DEV)
        moeq.grouped_matmul_fp8_block_epilogue(c, a, b, sa, sb, to_dev_u32(ro), to_dev_i32(ids),
                                               bias=bias, activation=act, residual=res)
        bad = ~torch.isfinite(c)
        want = torch.zeros_like(bad)
        want[:40, 5], want[40:, 7], want[3, 200], want[50, 100] = True, True, True, True
        assert torch.equal(bad, want)
        assert c[:40, 5].isnan().all() and (c[40:, 7] == inf).all()


def test_bad_groups_are_skipped():
    ro, ids, T, E, ins = _case([40, 30, 20], None, 128, 256, 0)
    a, b, sa, sb = (t.to(DEV) for t in ins)
    dc = synth.bf16_normal((T, 128), 1.0, seed=5, device=DEV)
    for off, eid, bits, live in (
            (ro, [0, 9, 2], moeq.DEVERR_BAD_EXPERT, [(0, 40), (70, 90)]),
            (ro, [0, -1, 2], moeq.DEVERR_BAD_EXPERT, [(0, 40), (70, 90)]),
            ([0, 40, 30, 90], [0, 1, 2], moeq.DEVERR_BAD_OFFSETS, [(0, 90)]),
            ([0, 40, 70, 91], [0, 1, 2], moeq.DEVERR_BAD_OFFSETS, [(0, 70)])):
        o, i = to_dev_u32(np.array(off)), to_dev_i32(np.array(eid))
        c = torch.full((T, 128), 7.0, dtype=BF16, device=DEV)
        dz, db = c.clone(), torch.full((E, 128), 7.0, device=DEV)
        moeq.grouped_matmul_fp8_block_epilogue(c, a, b, sa, sb, o, i, activation="silu")
        assert moeq.get_device_error() == bits
        moeq.clear_device_error()
        moeq.grouped_epilogue_grad(dc, o, i, E, d_z=dz, d_bias=db)
        assert moeq.get_device_error() == bits
        moeq.clear_device_error()
        rows = torch.zeros(T, dtype=torch.bool, device=DEV)
        for r0, r1 in live:
            rows[r0:r1] = True
        assert (c[~rows] == 7).all() and (dz[~rows] == 7).all()
        assert torch.equal(dz[rows], dc[rows]) and torch.isfinite(db).all()


# --------------------------------------------------------------- gradient

GROUPS = [([1], None, 16, 0), ([0, 3, 0, 70], [1, 0, 1, 2], 272, 3), ([127, 128, 129, 1], [1, 1, 0, 3], 144, 4),
          ([700], None, 1040, 0), ([5, 300, 0, 2], [0, 2, 1, 0], 2064, 9)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("counts,ids,N,tail", GROUPS)
def test_gradient_against_oracle(counts, ids, N, tail, act):
    ro, ids = groups_from_counts(counts, ids)
    T, E = int(ro[-1]) + tail, int(max(ids)) + 2           # an expert that no group has
    big = synth.bf16_normal((T, N + 8), 0.1, seed=1, device=DEV)
    dc, z = big[:, :N], synth.bf16_normal((T, N), 2.0, seed=2, device=DEV)
    if act is None:
        z = None
    new = lambda *s, dtype=torch.float32: torch.full(s, 7, dtype=dtype, device=DEV)      # noqa: E731
    q, s = new(T, N, dtype=torch.uint8), new(T, (N + 127) // 128)
    dz, db = new(T, N, dtype=BF16), new(E, N)
    off, eid = to_dev_u32(ro), to_dev_i32(ids)
    moeq.grouped_epilogue_grad(dc, off, eid, E, z=z, activation=act, q=q, scales=s, d_z=dz, d_bias=db)
    experts = L.row_experts(ro, ids, T)
    rows = experts >= 0
    ref, ref_db, mag = L.epilogue_grad(f64(dc), None if z is None else f64(z), act, experts, E)
    slope = 0.0 if act is None else 1.5e-6
    err = slope * np.abs(f64(dc)) + 2 * EPS * np.abs(ref)
    close(dz[rows], ref[rows], (err + U[BF16] * np.abs(ref))[rows])
    assert np.all(u8(q)[~rows] == 7) and (s[~rows] == 7).all() and (dz[~rows] == 7).all()
    total = np.zeros((E, N))
    for r in np.flatnonzero(rows):
        total[experts[r]] += slope * np.abs(f64(dc[r]))
    close(db, ref_db, (24 + T / 128 + 5) * EPS * mag + total + 1e-30)
    at = np.arange(N) // 128
    sv = f64(s)[rows]
    amax = np.stack([np.abs(ref[rows][:, at == i]).max(1) for i in range(sv.shape[1])], 1)
    amax_err = np.stack([err[rows][:, at == i].max(1) for i in range(sv.shape[1])], 1)
    assert np.all(np.abs(sv - amax / 448) <= amax_err / 448 + 2 * EPS * sv + 2.0 ** -126)
    off_by = np.abs(F.decode_e4m3(u8(q))[rows] * sv[:, at] - ref[rows])
    assert np.all(off_by <= 2.0 ** -4 * np.abs(ref[rows]) + 2.0 ** -10 * sv[:, at] + 1.1 * err[rows]
                  + 2.0 ** -120)
    if act is None:                                        # d_z is d_c: codes to the bit
        wq, ws = X.quantize_rows(dc.float().cpu().numpy()[rows])
        assert np.array_equal(u8(q)[rows], wq) and np.array_equal(s.cpu().numpy()[rows], ws)
    # each output alone is what it is with the others
    for kw in (dict(q=torch.zeros_like(q), scales=torch.zeros_like(s)), dict(d_z=torch.zeros_like(dz)),
               dict(d_bias=torch.zeros_like(db))):
        moeq.grouped_epilogue_grad(dc, off, eid, E, z=z, activation=act, **kw)
        for f, t in kw.items():
            full = dict(q=q, scales=s, d_z=dz, d_bias=db)[f]
            assert torch.equal(t, full) if f == "d_bias" else torch.equal(t[rows], full[rows])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_against_differences(act):
    z = np.linspace(-6, 6, 97)
    h = 1e-5
    diff = (L.activate(z + h, act)[0] - L.activate(z - h, act)[0]) / (2 * h)
    assert np.all(np.abs(L.activate(z, act)[1] - diff) < 1e-9)
    zt = torch.from_numpy(z).bfloat16().to(DEV)
    zt = torch.nn.functional.pad(zt, (0, 15)).view(1, -1).contiguous()
    one = torch.ones_like(zt)
    dz = torch.empty_like(zt)
    moeq.grouped_epilogue_grad(one, to_dev_u32([0, 1]), to_dev_i32([0]), 1, z=zt, activation=act, d_z=dz)
    close(dz, L.activate(f64(zt), act)[1], 1.5e-6 + U[BF16] * np.abs(L.activate(f64(zt), act)[1]))


def test_gradient_without_rows_and_many_groups():
    dc = torch.empty(0, 64, dtype=BF16, device=DEV)
    db = torch.full((3, 64), 7.0, device=DEV)
    moeq.grouped_epilogue_grad(dc, to_dev_u32([0, 0, 0]), to_dev_i32([0, 2]), 3, d_bias=db)
    assert not db.any()
    db.fill_(7.0)
    moeq.grouped_epilogue_grad(synth.bf16_normal((4, 64), 1.0, seed=1, device=DEV), to_dev_u32([0]),
                               torch.empty(0, dtype=torch.int32, device=DEV), 3, d_bias=db)
    assert not db.any()
    rng = np.random.default_rng(1)
    ro, ids = groups_from_counts(rng.integers(0, 6, 1024), rng.integers(0, 40, 1024))
    T = int(ro[-1])
    dc = synth.bf16_normal((T, 64), 1.0, seed=2, device=DEV)
    db = torch.zeros(40, 64, device=DEV)
    moeq.grouped_epilogue_grad(dc, to_dev_u32(ro), to_dev_i32(ids), 40, d_bias=db)
    _, ref, mag = L.epilogue_grad(f64(dc), None, None, L.row_experts(ro, ids, T), 40)
    close(db, ref, 200 * EPS * mag + 1e-30)                # some 26 groups an expert, of 5 rows at most


def test_gradient_of_many_rows_repeats_to_the_bit():
    """One expert's rows over many tiles; the same bits every time."""
    T, N = 40000, 272
    dc, z = synth.bf16_normal((T, N), 1.0, seed=3, device=DEV), synth.bf16_normal((T, N), 1.0, seed=4, device=DEV)
    off, eid = to_dev_u32([0, 39990]), to_dev_i32([0])
    out = []
    for _ in range(3):
        db = torch.zeros(1, N, device=DEV)
        moeq.grouped_epilogue_grad(dc, off, eid, 1, z=z, activation="gelu", d_bias=db)
        out.append(db)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    zd = z[:39990].double()
    slope = 0.5 * (1 + torch.erf(zd / 2 ** 0.5)) + zd * torch.exp(-0.5 * zd * zd) / (2 * np.pi) ** 0.5
    ref = (dc[:39990].double() * slope)
    tol = (24 + T / 128) * EPS * ref.abs().sum(0) + 1.5e-6 * dc.double().abs().sum(0)
    assert ((out[0][0].double() - ref.sum(0)).abs() <= tol).all()


# -------------------------------------------------- buffers, graphs, errors

@pytest.mark.parametrize("counts,N,K", [([0, 1, 127, 129, 3, 200], 272, 400), ([5, 90], 16, 16),
                                        ([1], 1008, 2720), ([130, 0, 2000, 4095], 528, 272)])
def test_stays_in_its_buffers(counts, N, K):
    ro, ids, T, E, ins = _case(counts, None, N, K, 0)
    a, b, sa, sb = (t.to(DEV) for t in _scaled(ins, 1.0))
    g = Guarded()
    off, eid = to_dev_u32(ro), to_dev_i32(ids)
    c, z = g((T, N), BF16), g((T, N), BF16)
    res = synth.bf16_normal((T, N), 1.0, seed=1, device=DEV)
    moeq.grouped_matmul_fp8_block_epilogue(c, a, b, sa, sb, off, eid, bias=torch.ones(E, N, device=DEV),
                                           activation="gelu", residual=res, z=z)
    G = len(ids)
    moeq.grouped_epilogue_grad(c, off, eid, E, z=z, activation="gelu", q=g((T, N), torch.uint8),
                               scales=g((T, (N + 127) // 128), torch.float32), d_z=g((T, N), BF16),
                               d_bias=g((E, N), torch.float32),
                               workspace=g((moeq.grouped_epilogue_grad_workspace(T, N, G),), torch.uint8))
    g.check()
    assert torch.isfinite(c.float()).all()


def test_streams_and_graphs():
    """On a given stream, and two graphs with workspaces of their own replayed at the
    same time."""
    N, K, counts = 528, 400, [300, 0, 500]
    ro, ids, T, E, ins = _case(counts, None, N, K, 0)
    a, b, sa, sb = (t.to(DEV) for t in _scaled(ins, 1.0))
    off, eid = to_dev_u32(ro), to_dev_i32(ids)
    bias = torch.ones(E, N, device=DEV)
    names = ("c", "z", "q", "scales", "d_z", "d_bias")

    def state(seed):
        new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device=DEV)             # noqa: E731
        return dict(res=synth.bf16_normal((T, N), 1.0, seed=seed, device=DEV), c=new(T, N), z=new(T, N),
                    q=new(T, N, dtype=torch.uint8), scales=new(T, 5, dtype=torch.float32), d_z=new(T, N),
                    d_bias=new(E, N, dtype=torch.float32),
                    ws=new(moeq.grouped_epilogue_grad_workspace(T, N, len(ids)), dtype=torch.uint8))

    def step(s, stream=None):
        moeq.grouped_matmul_fp8_block_epilogue(s["c"], a, b, sa, sb, off, eid, bias=bias, activation="silu",
                                               residual=s["res"], z=s["z"], stream=stream)
        moeq.grouped_epilogue_grad(s["c"], off, eid, E, z=s["z"], activation="silu", q=s["q"],
                                   scales=s["scales"], d_z=s["d_z"], d_bias=s["d_bias"],
                                   workspace=s["ws"], stream=stream)

    work, graphs, streams = [state(1), state(2)], [], [torch.cuda.Stream() for _ in range(2)]
    want = []
    for s, stream in zip(work, streams):
        step(s)
        torch.cuda.synchronize()
        want.append([s[f].clone() for f in names])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(s)
        graphs.append(graph)
        for f in names:
            s[f].zero_()
        torch.cuda.synchronize()
        step(s, stream=stream)
        stream.synchronize()
        assert all(torch.equal(s[f], w) for f, w in zip(names, want[-1]))
        for f in names:
            s[f].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for s, w in zip(work, want):
        assert all(torch.equal(s[f], v) for f, v in zip(names, w))


def test_refusals():
    T, N, K = 4, 64, 128
    c = torch.zeros(T, N, dtype=BF16, device=DEV)
    a, b = torch.zeros(T, K, dtype=torch.uint8, device=DEV), torch.zeros(1, N, K, dtype=torch.uint8, device=DEV)
    sa, sb = torch.ones(T, 1, device=DEV), torch.ones(1, 1, 1, device=DEV)
    off, eid = to_dev_u32([0, T]), to_dev_i32([0])
    args = (c, a, b, sa, sb, off, eid)
    for kw in (dict(activation="tanh"), dict(bias=torch.ones(N, device=DEV)), dict(residual=c.float()),
               dict(residual=c[:3]), dict(z=c.cpu()), dict(bias=torch.ones(1, N, dtype=BF16, device=DEV)),
               dict(num_active_experts=2)):
        with pytest.raises((ValueError, TypeError)):
            moeq.grouped_matmul_fp8_block_epilogue(*args, **kw)
    with pytest.raises(moeq.MoeqError):
        moeq.grouped_matmul_fp8_block_epilogue(*args, activation="silu", z=c)
    db = torch.zeros(1, N, device=DEV)
    for kw in (dict(activation="tanh", z=c, d_z=c), dict(q=a, scales=sa), dict(d_bias=db[0]),
               dict(d_bias=db, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)),
               dict(d_bias=db, stream=torch.cuda.Stream()), dict(num_active_experts=2, d_z=c)):
        with pytest.raises((ValueError, TypeError)):
            moeq.grouped_epilogue_grad(c, off, eid, 1, **kw)
    for kw in (dict(), dict(activation="silu", d_z=c.clone()), dict(z=c, d_z=c.clone())):
        with pytest.raises(moeq.MoeqError):
            moeq.grouped_epilogue_grad(c, off, eid, 1, **kw)
