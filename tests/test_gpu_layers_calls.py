"""The scored router, the norm and the product's epilogue as a program uses them: on a
stream of their own, in graphs, first calls from several threads, FP8 tensors by their
own type, offsets past 32 bits."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq, synth
from tests._util import DEV, need_gpu, to_dev_i32, to_dev_u32
from tests.test_gpu_experts import _gemm_inputs

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _error_word():
    need_gpu()
    moeq.clear_device_error()
    yield
    assert moeq.get_device_error() == 0


def _gate(T, E, seed, k=4):
    x = synth.uniform((T, E), -3, 3, seed=seed, device=DEV)
    b = synth.uniform((E,), -0.1, 0.1, seed=seed + 1, device=DEV)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    return x, b, ids, w, torch.empty(T, E, device=DEV)


def _gate_calls(x, b, ids, w, dx, stream=None):
    moeq.gate_group_topk(x, ids, w, bias=b, num_groups=4, topk_groups=2, stream=stream)
    moeq.gate_group_topk_grad(x, ids, w, dx, stream=stream)


def test_router_on_a_stream_and_in_a_graph():
    """A call waits for its own stream alone: the inputs arrive there."""
    want = _gate(5000, 64, 1)
    _gate_calls(*want)
    late = _gate(5000, 64, 1)
    src = [t.clone() for t in late[:2]]
    late[0].zero_()
    late[1].zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
        late[0].copy_(src[0])
        late[1].copy_(src[1])
    _gate_calls(*late, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, late))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        _gate_calls(*late)
    for seed in (3, 5):
        new = _gate(5000, 64, seed)
        _gate_calls(*new)
        late[0].copy_(new[0])
        late[1].copy_(new[1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(new, late))


def test_fp8_tensors_by_their_type():
    """uint8 and float8_e4m3fn buffers are the same codes."""
    T, K, N = 40, 256, 144
    x, w = synth.bf16_normal((T, K), 1.0, seed=1, device=DEV), torch.ones(K, dtype=BF16, device=DEV)
    s = [torch.empty(T, 2, device=DEV) for _ in range(2)]
    q = [torch.empty(T, K, dtype=d, device=DEV) for d in (torch.uint8, F8)]
    for a, b in zip(q, s):
        moeq.add_rms_norm(x, w, q=a, scales=b)
    assert torch.equal(q[0], q[1].view(torch.uint8)) and torch.equal(*s)
    _, b, _, sb = (t.to(DEV) for t in _gemm_inputs(1, 1, N, K, seed=1))
    off, ids = to_dev_u32([0, T]), to_dev_i32([0])
    c = [torch.empty(T, N, dtype=BF16, device=DEV) for _ in range(2)]
    for a, o, wt in zip(q, c, (b.view(torch.uint8), b.view(F8))):
        moeq.grouped_matmul_fp8_block_epilogue(o, a, wt, s[0], sb, off, ids, activation="relu")
    assert torch.equal(*c)
    g = [torch.empty(T, N, dtype=d, device=DEV) for d in (torch.uint8, F8)]
    for a, t in zip(g, s):
        moeq.grouped_epilogue_grad(c[0], off, ids, 1, z=c[0], activation="gelu", q=a, scales=t)
    assert torch.equal(g[0], g[1].view(torch.uint8))


def test_single_rows_of_any_stride():
    """A single row's stride says nothing."""
    big = synth.bf16_normal((3, 4096), 1.0, seed=2, device=DEV)
    row = big[1:2, :1000].as_strided((1, 1000), (7, 1))
    w = torch.ones(1000, dtype=BF16, device=DEV)
    y, z = (torch.empty(1, 1000, dtype=BF16, device=DEV) for _ in range(2))
    moeq.add_rms_norm(row.contiguous(), w, y=y)
    moeq.add_rms_norm(big[:1, :1000].as_strided((1, 1000), (7, 1), 4096), w, y=z)
    assert torch.equal(y, z)


def test_router_offsets_past_32_bits():
    T, E = (1 << 32) // (4 * 128) + 5000, 128              # 4.3 GB of logits
    x = torch.empty(T, E, device=DEV)
    few = synth.uniform((1000, E), -3, 3, seed=4, device=DEV)
    n = (T + 999) // 1000
    x.copy_(few.repeat(n, 1)[:T])
    ids, w = torch.empty(T, 6, dtype=torch.int32, device=DEV), torch.empty(T, 6, device=DEV)
    dx = torch.empty_like(x)
    b = synth.uniform((E,), -0.1, 0.1, seed=5, device=DEV)
    moeq.gate_group_topk(x, ids, w, bias=b, num_groups=8, topk_groups=4)
    moeq.gate_group_topk_grad(x, ids, w, dx)
    at = T // 1000 * 1000
    for t in (ids, w, dx):
        first = t[:1000].clone()
        assert torch.equal(t[:at].view(-1, 1000, t.shape[1]), first.expand(at // 1000, -1, -1))
        assert torch.equal(t[at:], first[:T - at])


def test_epilogue_offsets_past_32_bits():
    T, N, K = (1 << 32) // 8192 + 777, 8192, 16            # 8.6 GB of bf16 each
    a, b, sa, sb = (t.to(DEV) for t in _gemm_inputs(512, 1, N, K, seed=6))
    reps = (T + 511) // 512
    many, scales = a.repeat(reps, 1)[:T].contiguous(), sa.repeat(reps, 1)[:T].contiguous()
    bias, ids = torch.ones(1, N, device=DEV), to_dev_i32([0])
    few = torch.ones(512, N, dtype=BF16, device=DEV)
    moeq.grouped_matmul_fp8_block_epilogue(few, a, b, sa, sb, to_dev_u32([0, 512]), ids, bias=bias,
                                           activation="silu", residual=few)
    c = torch.ones(T, N, dtype=BF16, device=DEV)
    off = to_dev_u32([0, T])
    moeq.grouped_matmul_fp8_block_epilogue(c, many, b, scales, sb, off, ids, bias=bias,
                                           activation="silu", residual=c)
    for r in range(0, T, 1 << 16):
        rows = torch.arange(r, min(T, r + (1 << 16)), device=DEV) % 512
        assert torch.equal(c[r:r + (1 << 16)], few[rows])
    fq, fs = torch.empty(512, N, dtype=torch.uint8, device=DEV), torch.empty(512, N // 128, device=DEV)
    moeq.grouped_epilogue_grad(few, to_dev_u32([0, 512]), ids, 1, z=few, activation="gelu_tanh", q=fq, scales=fs)
    q, s = torch.empty(T, N, dtype=torch.uint8, device=DEV), torch.empty(T, N // 128, device=DEV)
    db = torch.empty(1, N, device=DEV)
    moeq.grouped_epilogue_grad(c, off, ids, 1, z=c, activation="gelu_tanh", q=q, scales=s, d_bias=db)
    for r in range(0, T, 1 << 16):
        rows = torch.arange(r, min(T, r + (1 << 16)), device=DEV) % 512
        assert torch.equal(q[r:r + (1 << 16)], fq[rows]) and torch.equal(s[r:r + (1 << 16)], fs[rows])
    assert torch.isfinite(db).all()


THREADS = """
    import sys, threading
    sys.path.insert(0, sys.argv[1])
    import torch
    from fp4_fp8_quantization_gb300 import moeq, synth
    T, K, N, E = 300, 256, 272, 2
    x = synth.bf16_normal((T, K), 1.0, seed=1, device="cuda")
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    wq = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    ws = torch.ones(E, 3, 2, device="cuda")
    off = torch.tensor([0, 100, T], dtype=torch.int32, device="cuda")
    ids = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    bias = torch.ones(E, N, device="cuda")
    torch.cuda.synchronize()
    out, gate = [None] * 8, threading.Barrier(8)
    def go(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            new = lambda *a, dtype=torch.float32: torch.zeros(a, dtype=dtype, device="cuda")
            q, sc, u, h = new(T, K, dtype=torch.uint8), new(T, 2), new(T), new(T, K, dtype=torch.bfloat16)
            c, z = new(T, N, dtype=torch.bfloat16), new(T, N, dtype=torch.bfloat16)
            g, gs, db = new(T, N, dtype=torch.uint8), new(T, 3), new(E, N)
            ti, tw, dx, dw = new(T, 4, dtype=torch.int32), new(T, 4), new(T, K, dtype=torch.bfloat16), new(K)
            gate.wait()
            moeq.add_rms_norm(x, w, residual=x, h=h, q=q, scales=sc, rstd=u)
            moeq.grouped_matmul_fp8_block_epilogue(c, q, wq, sc, ws, off, ids, bias=bias, activation="gelu", z=z)
            moeq.grouped_epilogue_grad(c, off, ids, E, z=z, activation="gelu", q=g, scales=gs, d_bias=db)
            moeq.gate_group_topk(h, ti, tw, num_groups=8, topk_groups=3)
            moeq.add_rms_norm_grad(x, h, w, u, dx, d_weight=dw)
        s.synchronize()
        out[i] = [t.cpu() for t in (q, sc, c, z, g, gs, db, ti, tw, dx, dw)]
    ts = [threading.Thread(target=go, args=(i,)) for i in range(8)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert moeq.get_device_error() == 0
    assert all(torch.equal(a, b) for o in out[1:] for a, b in zip(out[0], o))
    print("THREADS OK")
"""


def test_first_calls_from_threads():
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(THREADS), ROOT], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "THREADS OK" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
