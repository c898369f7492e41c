"""The activations' gradient of the FP8 block GEMM: the same call on transposed
weights."""
import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq, synth
from oracle import formats as F
from tests._util import DEV, assert_gemm_close, bf16_bits, groups_from_counts, need_gpu, u8
from tests.test_gpu_experts import _gemm, _gemm_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,ids,N,K", [
    ([3, 0, 40, 129], [1, 0, 2, 0], 144, 200), ([300, 128, 33], [0, 2, 1], 528, 1160),
    ([2100, 1900, 0, 2003], [2, 0, 1, 3], 2608, 520)])
def test_block_gemm_gradient_on_transposed_weights(counts, ids, N, K):
    """The activations' gradient, d_a[t, k] = sum over n of d_c[t, n] b[e, n, k],
    is the same call with the weights' codes and scales transposed."""
    need_gpu()
    moeq.clear_device_error()
    ro, ids = groups_from_counts(counts, ids)
    n, E2 = int(ro[-1]), max(ids) + 1
    _, b, _, sb = _gemm_inputs(1, E2, N, K, seed=N)
    d_c = synth.bf16_normal((n, N), 1.0, seed=K)
    q = torch.empty((n, N), dtype=torch.uint8, device=DEV)
    s = torch.empty((n, (N + 127) // 128), device=DEV)
    moeq.quantize_fp8_block(d_c.to(DEV), q, s)
    bt = b.view(torch.uint8).transpose(1, 2).contiguous().view(torch.float8_e4m3fn)
    d_a = _gemm(q.cpu().view(torch.float8_e4m3fn), bt, s.cpu(), sb.transpose(1, 2).contiguous(), ro, ids)
    # from the weights as they were
    deq = (F.decode_e4m3(u8(b)) * sb.double().numpy()[:, np.arange(N) // 128][:, :, np.arange(K) // 128])
    dq = F.decode_e4m3(u8(q)) * s.double().cpu().numpy()[:, np.arange(N) // 128]
    want = np.zeros((n, K))
    for g, e in enumerate(ids):
        want[ro[g]:ro[g + 1]] = dq[ro[g]:ro[g + 1]] @ deq[e]
    assert_gemm_close(bf16_bits(d_a), want)
    assert moeq.get_device_error() == 0
