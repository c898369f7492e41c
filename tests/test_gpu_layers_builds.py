"""The scored router, the norm and the product's epilogue in the test builds of the
library: every store checked by address, each tile of the product for every size,
and a pipeline stage that never loads."""
import os
import subprocess
import sys

import pytest

from fp4_fp8_quantization_gb300 import moeq
from tests._util import need_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _pytest(lib, *args, **env):
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", *args],
                       cwd=ROOT, env=dict(os.environ, MOEQ_LIB=lib, **env), capture_output=True,
                       text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout


def test_debug_bounds_build_flags_no_store(tmp_path):
    need_gpu()
    from fp4_fp8_quantization_gb300 import build
    lib = build.build(out_dir=str(tmp_path), defines=["MOEQ_DEBUG_BOUNDS"])
    _pytest(lib, "tests/test_gpu_gate_group.py", "tests/test_gpu_norm.py", "tests/test_gpu_epilogue.py",
            "-k", "stays or many_tokens or product_against or gradient_against_oracle",
            MOEQ_CHECK_BOUNDS="1")


@pytest.mark.parametrize("tile", [0, 1, 2])
def test_epilogue_on_each_tile(tmp_path, tile):
    need_gpu()
    from fp4_fp8_quantization_gb300 import build
    lib = build.build(out_dir=str(tmp_path), defines=[f"MOEQ_FP8_BLOCK_TILE={tile}"])
    _pytest(lib, "tests/test_gpu_epilogue.py", "-k",
            "product_against or plain_product or nonfinite or bad_groups or stays")


CHILD = r"""
import sys, time
import torch
sys.path.insert(0, sys.argv[1])
from fp4_fp8_quantization_gb300 import moeq, synth
dev, rows, K, N = "cuda", int(sys.argv[2]), 1024, 384
a = synth.e4m3_normal((rows, K), 50.0, seed=1, device=dev)
b = synth.e4m3_normal((2, N, K), 50.0, seed=2, device=dev)
sa, sb = torch.ones(rows, 8, device=dev), torch.ones(2, 3, 8, device=dev)
c, res = (torch.zeros(rows, N, dtype=torch.bfloat16, device=dev) for _ in range(2))
ro = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device=dev)
ids = torch.tensor([1, 0], dtype=torch.int32, device=dev)
moeq.clear_device_error()
t0 = time.time()
moeq.grouped_matmul_fp8_block_epilogue(c, a, b, sa, sb, ro, ids, bias=torch.ones(2, N, device=dev),
                                       activation="silu", residual=res,
                                       z=torch.empty_like(c) if int(sys.argv[3]) else None)
torch.cuda.synchronize()
dt = time.time() - t0
bits = moeq.get_device_error()
moeq.clear_device_error()
x = torch.arange(1 << 20, device=dev, dtype=torch.int64)
print("RESULT", bits, moeq.get_device_error(), int(x.sum()) == (1 << 20) * ((1 << 20) - 1) // 2, dt)
"""


@pytest.fixture(scope="module")
def stuck(tmp_path_factory):
    need_gpu()
    from fp4_fp8_quantization_gb300 import build
    return build.build(out_dir=str(tmp_path_factory.mktemp("stuck")), defines=["MOEQ_TEST_STUCK_STAGE"])


@pytest.mark.parametrize("rows,saved", [(12, True), (6000, True), (6000, False)])
def test_stuck_stage_times_out_and_context_survives(stuck, rows, saved):
    """The bounded waits run out in each form, the kernel reports it and leaves."""
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, str(rows), str(int(saved))], cwd=ROOT,
                       env=dict(os.environ, MOEQ_LIB=stuck), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    line = [ln for ln in r.stdout.splitlines() if ln.startswith("RESULT")][-1].split()
    assert int(line[1]) & moeq.DEVERR_TIMEOUT and int(line[2]) == 0
    assert line[3] == "True" and float(line[4]) < 30
