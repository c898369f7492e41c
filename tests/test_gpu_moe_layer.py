"""The example layer, serving and training, and the FP8-block kernels in the
test builds of the library (store bounds checked; a stage that never loads)."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq
from tests._util import DEV, need_gpu, note

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "moe_layer_example", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_serves():
    # E4M3 keeps 3 mantissa bits: 2^-4 relative at most per operand, 2^-4 / sqrt(3)
    # in the root mean square.  Four quantized operands meet (two products, the
    # second's input passing through SwiGLU), with independent errors: below
    # 2 * sqrt(4) * 2^-4 / sqrt(3).  The routed choices agree up to near-ties.
    need_gpu()
    many, one = _example().serve()
    note(many=many, one=one)
    assert many < 0.15 and one < 0.15


def test_example_learns():
    need_gpu()
    first, last = _example().train()
    note(first=first, last=last)
    assert last < 0.5 * first


def test_autograd_functions_against_plain_autograd():
    """The layer's gradients in fp32 against autograd through the definition:
    three products of length H or 2 I in fp32 on both sides, 2^-24 each term."""
    need_gpu()
    m = _example()
    T, E, H, I, k = 40, 6, 64, 32, 3
    params = [w.float() for w in m.make_weights(E, H, I, seed=7)]
    x = torch.randn(T, H, device=DEV, generator=torch.Generator(DEV).manual_seed(8))
    up = torch.randn(T, H, device=DEV, generator=torch.Generator(DEV).manual_seed(9))
    grads = []
    for f in (m.trained_layer, m.plain_layer):
        leaves = [t.clone().requires_grad_() for t in [x, *params]]
        (f(leaves[0], *leaves[1:], k) * up).sum().backward()
        grads.append([t.grad for t in leaves])
    for a, b in zip(*grads):
        assert float((a - b).norm() / b.norm()) < 1e-5   # ~ sqrt(H) 2^-24 and the router's exp
    assert moeq.get_device_error() == 0


def test_debug_bounds_build_flags_no_store(tmp_path):
    need_gpu()
    from fp4_fp8_quantization_gb300 import build
    lib = build.build(out_dir=str(tmp_path), defines=["MOEQ_DEBUG_BOUNDS"])
    env = dict(os.environ, MOEQ_LIB=lib, MOEQ_CHECK_BOUNDS="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        "tests/test_gpu_experts.py", "-k",
                        "against_oracle or gradients or bit_exact or many_tokens or layer"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout


CHILD = r"""
import sys, time
import torch
sys.path.insert(0, sys.argv[1])
from fp4_fp8_quantization_gb300 import moeq, synth
dev, rows, K, N = "cuda", int(sys.argv[2]), int(sys.argv[3]), 384
a = synth.e4m3_normal((rows, K), 50.0, seed=1, device=dev)
b = synth.e4m3_normal((2, N, K), 50.0, seed=2, device=dev)
sa = torch.ones(rows, (K + 127) // 128, device=dev)
sb = torch.ones(2, (N + 127) // 128, (K + 127) // 128, device=dev)
c = torch.zeros(rows, N, dtype=torch.bfloat16, device=dev)
ro = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device=dev)
ids = torch.tensor([1, 0], dtype=torch.int32, device=dev)
moeq.clear_device_error()
t0 = time.time()
moeq.grouped_matmul_fp8_block(c, a, b, sa, sb, ro, ids)
torch.cuda.synchronize()
dt = time.time() - t0
bits = moeq.get_device_error()
moeq.clear_device_error()
x = torch.arange(1 << 20, device=dev, dtype=torch.int64)
print("RESULT", bits, moeq.get_device_error(), int(x.sum()) == (1 << 20) * ((1 << 20) - 1) // 2, dt)
"""


@pytest.mark.parametrize("rows,K", [(12, 1024), (6000, 1024), (6000, 3200)])
def test_stuck_stage_times_out_and_context_survives(tmp_path, rows, K):
    """A stage that is announced and never loaded, in each tile shape: the
    bounded waits run out, the kernel reports it and leaves."""
    need_gpu()
    from fp4_fp8_quantization_gb300 import build
    lib = build.build(out_dir=str(tmp_path), defines=["MOEQ_TEST_STUCK_STAGE"])
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, str(rows), str(K)], cwd=ROOT,
                       env=dict(os.environ, MOEQ_LIB=lib), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    line = [ln for ln in r.stdout.splitlines() if ln.startswith("RESULT")][-1].split()
    assert int(line[1]) & moeq.DEVERR_TIMEOUT and int(line[2]) == 0
    assert line[3] == "True" and float(line[4]) < 30
