"""Stores of the router, row, FP8-block and FP8-block GEMM calls stay in their
buffers: every output between canary guards, and the debug build that checks
each store's addresses, on the sizes of both GEMM tiles and of every kernel's
forms."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq, synth
from tests._util import DEV, groups_from_counts, need_gpu, to_dev_i32, to_dev_u32
from tests.test_gpu_experts import _dst, _gemm_inputs
from tests.test_gpu_guard_regions import Guarded

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _error_word():
    need_gpu()
    moeq.clear_device_error()
    yield
    assert moeq.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 7), (8193, 30, 5), (8195, 61, 8),
                                   (16387, 127, 11), (33, 129, 9), (9, 1023, 32), (3, 8, 8)])
@pytest.mark.parametrize("normalize", [False, True])
def test_router_stays_in_its_buffers(T, E, k, normalize, dtype):
    g = Guarded()
    x = synth.bf16_normal((T, E), 2.0, seed=T, device=DEV).to(dtype)
    ids, w = g((T, k), torch.int32), g((T, k), torch.float32)
    dx = g((T, E), dtype)
    moeq.gate_topk(x, ids, w, normalize=normalize)
    moeq.gate_topk_grad(x, ids, torch.ones(T, k, device=DEV), dx, normalize=normalize)
    g.check()
    assert torch.isfinite(w).all() and torch.isfinite(dx.float()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (37, 120, 4), (301, 776, 2), (130, 1544, 8),
                                   (7, 7176, 8), (33, 64, 11), (5, 2056, 20)])
def test_row_calls_stay_in_their_buffers(T, H, k, dtype):
    rng = np.random.default_rng(H)
    R = T * k
    g = Guarded()
    dst = torch.from_numpy(_dst(T, k, R, rng)).to(DEV)
    x = synth.bf16_normal((T, H), 1.0, seed=1, device=DEV).to(dtype)
    rows = synth.bf16_normal((R, H), 1.0, seed=2, device=DEV).to(dtype)
    w = synth.uniform((T, k), 0.1, 1.0, seed=3, device=DEV)
    moeq.permute_topk(x, dst, g((R, H), dtype), weights=w)
    moeq.permute_topk_grad(rows, dst, g((T, H), dtype), weights=w, tokens=x,
                           d_weights=g((T, k), torch.float32))
    moeq.combine_topk(rows, dst, g((T, H), dtype), weights=w)
    moeq.combine_topk_grad(x, dst, g((R, H), dtype), weights=w, rows=rows,
                           d_weights=g((T, k), torch.float32))
    g.check()


@pytest.mark.parametrize("T,K,k", [(1, 16, 1), (3, 144, 2), (33, 272, 8), (7, 1040, 3),
                                   (129, 2064, 4), (5, 4112, 20)])
def test_block_quantizers_stay_in_their_buffers(T, K, k):
    rng = np.random.default_rng(K)
    kb, g = (K + 127) // 128, Guarded()
    u8, f32 = torch.uint8, torch.float32
    x = synth.bf16_normal((T, 2 * K), 1.0, seed=K, device=DEV)
    moeq.quantize_fp8_block(x[:, :K], g((T, K), u8), g((T, kb), f32))
    dst = torch.from_numpy(_dst(T, k, T * k, rng)).to(DEV)
    moeq.quantize_fp8_block_topk(x[:, :K], dst, g((T * k, K), u8), g((T * k, kb), f32))
    moeq.swiglu_quantize_fp8_block(x, g((T, K), u8), g((T, kb), f32))
    wt = synth.bf16_normal((2, T, K), 1.0, seed=K + 1, device=DEV)
    moeq.quantize_fp8_block_weight(wt, g((2, T, K), u8), g((2, (T + 127) // 128, kb), f32))
    g.check()


def test_large_swiglu_quantizer_stays_in_its_buffers():
    R, I = 32801, 1040                       # past 2^25 values: the table form
    g = Guarded()
    y = synth.bf16_normal((R, 2 * I), 1.0, seed=1, device=DEV)
    moeq.swiglu_quantize_fp8_block(y, g((R, I), torch.uint8), g((R, 9), torch.float32))
    g.check()


@pytest.mark.parametrize("counts,N,K", [
    ([0, 1, 127, 129, 3, 200], 264, 400), ([5, 90], 8, 16), ([1], 1000, 2720),
    ([128] * 32 + [4], 520, 272), ([130, 0, 2000, 4095], 520, 2720)])
def test_block_gemm_stays_in_its_buffer(counts, N, K):
    ro, ids = groups_from_counts(counts)
    T, E = int(ro[-1]), len(counts)
    a, b, sa, sb = (t.to(DEV) for t in _gemm_inputs(T, E, N, K, seed=7))
    g = Guarded()
    c = g((T, N), torch.bfloat16)
    moeq.grouped_matmul_fp8_block(c, a, b, sa, sb, to_dev_u32(ro), to_dev_i32(ids))
    g.check()
    assert torch.isfinite(c.float()).all()


def test_debug_bounds_build_flags_no_store_of_any_form(tmp_path):
    """The build that checks each store's addresses, on the large tiles too."""
    from fp4_fp8_quantization_gb300 import build
    lib = build.build(out_dir=str(tmp_path), defines=["MOEQ_DEBUG_BOUNDS"])
    env = dict(os.environ, MOEQ_LIB=lib, MOEQ_CHECK_BOUNDS="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        "tests/test_gpu_experts_tiles.py", "tests/test_gpu_experts_guards.py",
                        "-k", "against_oracle or stays or stay_in"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
