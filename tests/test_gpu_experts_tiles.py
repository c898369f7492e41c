"""The FP8 block GEMM at sizes that take its 128 x 256 tiles, against the
float64 oracle: both forms (results stored directly, or by tensor stores during
the next tile), full and partial 128-row blocks, group ends inside and at the
32-row boxes, empty groups, last tiles with 8 to 136 columns, CTAs with several
tiles, K that ends inside a block.

The GEMM chooses its form by a rule on the sizes.  So that no change of the rule
takes a form out of the tests, all GEMM tests, these and those of
test_gpu_experts, also run on three builds of the library that know one form
each (MOEQ_FP8_BLOCK_TILE).  Tolerances as in test_gpu_experts."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq
from oracle import experts as X
from tests._util import assert_gemm_close, bf16_bits, groups_from_counts, need_gpu, u8
from tests.test_gpu_experts import CANARY, _gemm, _gemm_inputs

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# 6904 rows: blocks of exactly 128 and of one row more, ends on and off the boxes
RAGGED = [0, 128, 1, 257, 640, 31, 2000, 33, 0, 1185, 96, 1500, 129, 3, 900, 1]
IDS = [3, 5, 0, 2, 1, 4, 6, 0, 7, 3, 5, 1, 2, 6, 4, 7]     # experts with two groups


@pytest.fixture(autouse=True)
def _error_word():
    need_gpu()
    moeq.clear_device_error()
    yield


@pytest.mark.parametrize("counts,ids,N,K,tail", [
    (RAGGED, IDS, 520, 400, 5),
    (RAGGED, IDS, 648, 2560, 0),
    ([12300], [1], 1032, 144, 3),               # four tiles per CTA
    (list(range(60, 124)), None, 1000, 1024, 0),
    (RAGGED, IDS, 648, 2576, 0),
    (RAGGED, IDS, 520, 2720, 5),
    ([4100, 0, 4000, 127], [1, 0, 0, 2], 1032, 3200, 1),
    (list(range(60, 124)), None, 1000, 2816, 0),
])
def test_large_tiles_against_oracle(counts, ids, N, K, tail):
    ro, ids = groups_from_counts(counts, ids)
    n, E = int(ro[-1]), int(max(ids)) + 1
    a, b, sa, sb = _gemm_inputs(n + tail, E, N, K, seed=N + K)
    c = _gemm(a, b, sa, sb, ro, ids)
    ref = X.matmul(u8(a), u8(b), sa.numpy(), sb.numpy(), ro, ids)
    assert_gemm_close(bf16_bits(c)[:n], ref[:n])
    assert bool((c[n:] == CANARY).all())
    assert moeq.get_device_error() == 0


@pytest.mark.parametrize("K", [400, 2720])
def test_large_tiles_scales_are_exact_powers(K):
    """As test_block_gemm_scales_are_exact_powers: rescaling both sides of one
    K block, one row and one column block shifts exponents only."""
    ro, ids = groups_from_counts(RAGGED, IDS)
    a, b, sa, sb = _gemm_inputs(int(ro[-1]), 8, 520, K, seed=5)
    sa, sb = torch.full_like(sa, 0.5), torch.full_like(sb, 0.25)
    c = _gemm(a, b, sa, sb, ro, ids).float()
    row = int(ro[6]) + 130                                  # the second block of 2000 rows
    sa[row] *= 4.0
    sb[6, 1] *= 8.0
    want = c.clone()
    want[row] *= 4.0
    for g, e in enumerate(ids):
        if e == 6:
            want[int(ro[g]):int(ro[g + 1]), 128:256] *= 8.0
    assert torch.equal(_gemm(a, b, sa, sb, ro, ids).float(), want)
    sa[:, 1] *= 2.0 ** -7
    sb[:, :, 1] *= 2.0 ** 7
    assert torch.equal(_gemm(a, b, sa, sb, ro, ids).float(), want)


@pytest.mark.parametrize("K", [400, 2720])
def test_large_tiles_keep_nonfinite_values_in_their_row_and_column(K):
    ro, ids = groups_from_counts(RAGGED, IDS)
    a, b, sa, sb = _gemm_inputs(int(ro[-1]), 8, 520, K, seed=9)
    clean = _gemm(a, b, sa, sb, ro, ids)
    ab, bb, sa2 = a.view(torch.uint8).clone(), b.view(torch.uint8).clone(), sa.clone()
    rows = [int(ro[6]) + 127, int(ro[9]) + 1184]            # a block's end, a group's end
    ab[rows, K - 1] = 0x7F
    bb[2, 513, 5] = 0xFF                                    # in the last column tile
    sa2[int(ro[11]) + 700, 1] = float("inf")
    got = _gemm(ab.view(torch.float8_e4m3fn), bb.view(torch.float8_e4m3fn), sa2, sb, ro, ids)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[rows], bad[int(ro[11]) + 700] = True, True
    for g, e in enumerate(ids):
        if e == 2:
            bad[int(ro[g]):int(ro[g + 1]), 513] = True
    assert not torch.isfinite(got[bad]).any()
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("K", [400, 2720])
def test_large_tiles_skip_bad_groups(K):
    ro, ids = groups_from_counts(RAGGED, IDS)
    n = int(ro[-1])
    a, b, sa, sb = _gemm_inputs(n, 8, 520, K, seed=3)
    good = _gemm(a, b, sa, sb, ro, ids)
    bad_ids = ids.copy()
    bad_ids[6] = 8
    c = _gemm(a, b, sa, sb, ro, bad_ids)
    assert moeq.get_device_error() == moeq.DEVERR_BAD_EXPERT
    keep = np.ones(n, bool)
    keep[int(ro[6]):int(ro[7])] = False
    keep = torch.from_numpy(keep).to(c.device)
    assert torch.equal(c[keep], good[keep]) and bool((c[~keep] == CANARY).all())
    moeq.clear_device_error()
    bad_ro = ro.copy()
    bad_ro[16] = n + 1                                      # the last group ends past the rows
    c = _gemm(a, b, sa, sb, bad_ro, ids)
    assert moeq.get_device_error() == moeq.DEVERR_BAD_OFFSETS
    assert torch.equal(c[:n - 1], good[:n - 1]) and bool((c[n - 1:] == CANARY).all())
    moeq.clear_device_error()


@pytest.mark.parametrize("tile", [0, 1, 2])
def test_build_of_one_form_passes_the_gemm_tests(tmp_path, tile):
    from fp4_fp8_quantization_gb300 import build
    lib = build.build(out_dir=str(tmp_path), defines=[f"MOEQ_FP8_BLOCK_TILE={tile}"])
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        "tests/test_gpu_experts.py", "tests/test_gpu_experts_tiles.py",
                        "-k", "block_gemm or large_tiles or cuda_graph"],
                       cwd=ROOT, env=dict(os.environ, MOEQ_LIB=lib), capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
