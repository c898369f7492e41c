"""The router, row, FP8-block and FP8-block GEMM calls as a program uses them:
each on a stream of its own, and first calls from several threads."""
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


@pytest.fixture(autouse=True)
def _error_word():
    need_gpu()
    moeq.clear_device_error()
    yield
    assert moeq.get_device_error() == 0


# ----------------------------------------------------------------- streams

T, E, K, H = 64, 32, 4, 256
R = T * K


def _out(shape, dtype=torch.float32):
    return torch.full(shape, 7, dtype=dtype, device=DEV)


def _gate_fwd(v, s):
    out = _out((T, K), torch.int32), _out((T, K))
    moeq.gate_topk(v["logits"], *out, stream=s)
    return out


def _gate_bwd(v, s):
    out = _out((T, E))
    moeq.gate_topk_grad(v["logits"], v["ids"], v["dw"], out, normalize=False, stream=s)
    return out,


def _permute(v, s):
    out = _out((R, H), torch.bfloat16)
    moeq.permute_topk(v["x"], v["dst"], out, weights=v["dw"], stream=s)
    return out,


def _permute_grad(v, s):
    out = _out((T, H), torch.bfloat16), _out((T, K))
    moeq.permute_topk_grad(v["rows"], v["dst"], out[0], weights=v["dw"], tokens=v["x"],
                           d_weights=out[1], stream=s)
    return out


def _combine(v, s):
    out = _out((T, H), torch.bfloat16)
    moeq.combine_topk(v["rows"], v["dst"], out, weights=v["dw"], stream=s)
    return out,


def _combine_grad(v, s):
    out = _out((R, H), torch.bfloat16), _out((T, K))
    moeq.combine_topk_grad(v["x"], v["dst"], out[0], weights=v["dw"], rows=v["rows"],
                           d_weights=out[1], stream=s)
    return out


def _quantize(v, s):
    out = _out((R, H), torch.uint8), _out((R, 2))
    moeq.quantize_fp8_block(v["rows"], *out, stream=s)
    return out


def _quantize_topk(v, s):
    out = _out((R, H), torch.uint8), _out((R, 2))
    moeq.quantize_fp8_block_topk(v["x"], v["dst"], *out, stream=s)
    return out


def _swiglu(v, s):
    out = _out((R, H // 2), torch.uint8), _out((R, 1))
    moeq.swiglu_quantize_fp8_block(v["rows"], *out, stream=s)
    return out


def _weight(v, s):
    out = _out((2, R // 2, H), torch.uint8), _out((2, 1, 2))
    moeq.quantize_fp8_block_weight(v["rows"].view(2, R // 2, H), *out, stream=s)
    return out


def _matmul(v, s):
    out = _out((R, 136), torch.bfloat16)
    moeq.grouped_matmul_fp8_block(out, v["a"], v["b"], v["sa"], v["sb"], v["offsets"], v["experts"],
                                  stream=s)
    return out,


CALLS = [_gate_fwd, _gate_bwd, _permute, _permute_grad, _combine, _combine_grad, _quantize,
         _quantize_topk, _swiglu, _weight, _matmul]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__[1:])
def test_each_call_runs_on_the_stream_it_is_given(call):
    """The values come to the inputs on that stream only, behind work that keeps
    it busy: a call on another stream would work on zeros."""
    a, b, sa, sb = _gemm_inputs(R, 2, 136, H, seed=1)
    real = dict(logits=synth.uniform((T, E), -3, 3, seed=2), dw=synth.uniform((T, K), 0.5, 2, seed=3),
                x=synth.bf16_normal((T, H), 1.0, seed=4), rows=synth.bf16_normal((R, H), 1.0, seed=5),
                a=a.view(torch.uint8), b=b.view(torch.uint8), sa=sa, sb=sb)
    real = {n: t.to(DEV) for n, t in real.items()}
    fixed = dict(dst=torch.arange(R, dtype=torch.int32, device=DEV).view(T, K),
                 ids=torch.arange(R, dtype=torch.int32, device=DEV).view(T, K) % E,
                 offsets=to_dev_u32([0, 100, R]), experts=to_dev_i32([1, 0]))
    want = call(dict(real, **fixed), None)
    late = {n: torch.zeros_like(t) for n, t in real.items()}
    zero = call(dict(late, **fixed), None)
    assert any(not torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(want, zero))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(8):
            big = (big @ big).clamp_(-1, 1)
        for n, t in late.items():
            t.copy_(real[n])
    got = call(dict(late, **fixed), s)
    s.synchronize()
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


# ----------------------------------------------------------------- threads

CHILD = textwrap.dedent("""
    import sys, threading
    import torch
    sys.path.insert(0, ROOT)
    from fp4_fp8_quantization_gb300 import moeq, synth
    torch.cuda.set_device(0)
    dev = "cuda"
    N, G = 520, 16
    sizes = [(40, 400), (6912, 400), (6912, 2720)]      # the three forms of the GEMM
    data = []
    for rows, k in sizes:
        kb = (k + 127) // 128
        data.append((synth.e4m3_normal((rows, k), 50.0, seed=1, device=dev),
                     synth.e4m3_normal((G, N, k), 50.0, seed=2, device=dev),
                     synth.uniform((rows, kb), 0.002, 0.02, seed=3, device=dev),
                     synth.uniform((G, 5, kb), 0.002, 0.02, seed=4, device=dev),
                     torch.arange(G + 1, dtype=torch.int32, device=dev) * rows // G))
    ids = torch.arange(G, dtype=torch.int32, device=dev)
    y = synth.bf16_normal((300, 512), 1.0, seed=5, device=dev)
    lg = synth.uniform((300, 64), -3, 3, seed=6, device=dev)
    torch.cuda.synchronize()

    def work(stream, first):
        out = []
        with torch.cuda.stream(stream):
            t, w = torch.zeros(300, 4, dtype=torch.int32, device=dev), torch.zeros(300, 4, device=dev)
            moeq.gate_topk(lg, t, w, stream=stream)
            q = torch.zeros(300, 256, dtype=torch.uint8, device=dev)
            s = torch.zeros(300, 2, device=dev)
            moeq.swiglu_quantize_fp8_block(y, q, s, stream=stream)
            for i in range(3):
                a, b, sa, sb, ro = data[(first + i) % 3]
                c = torch.zeros((a.shape[0], N), dtype=torch.bfloat16, device=dev)
                moeq.grouped_matmul_fp8_block(c, a, b, sa, sb, ro.int(), ids, stream=stream)
                out.append(((first + i) % 3, c))
        stream.synchronize()
        return [v.cpu() for v in (t, w, q, s)] + [c.cpu() for _, c in sorted(out, key=lambda p: p[0])]

    results = [None] * 8
    streams = [torch.cuda.Stream() for _ in range(8)]
    start = threading.Barrier(8)

    def run(i):
        start.wait()
        results[i] = work(streams[i], i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(8)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    ref = work(torch.cuda.Stream(), 0)
    for r in results:
        assert r is not None
        for got, want in zip(r, ref):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    assert moeq.get_device_error() == 0
    print("threads ok")
""")


def test_first_block_gemm_calls_from_eight_threads():
    """Kernel attributes are set up once per device and form: first calls made
    at the same time, in different orders of the forms, give the same bytes as
    later ones."""
    r = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + CHILD], capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "threads ok" in r.stdout
