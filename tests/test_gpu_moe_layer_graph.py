"""The example's serving layer with its workspaces, in a CUDA graph."""
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq, synth
from tests._util import DEV, need_gpu
from tests.test_gpu_moe_layer import _example

pytestmark = pytest.mark.gpu


def test_example_layer_in_a_cuda_graph():
    """Fp8MoeLayer with an output given allocates nothing after its first call,
    and replays in a graph with the bytes of the direct calls."""
    need_gpu()
    moeq.clear_device_error()
    m = _example()
    weights = m.make_weights(8, 256, 128, seed=1)
    layer = m.Fp8MoeLayer(*weights, top_k=2, max_tokens=96)
    x, out = (torch.empty(80, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    x.copy_(synth.bf16_normal((80, 256), 1.0, seed=2, device=DEV))
    assert layer(x, out) is out
    torch.cuda.synchronize()
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]           # noqa: E731
    before = count()
    layer(x, out)
    assert count() == before
    side = torch.cuda.Stream()                       # cuBLAS has a workspace for each stream
    with torch.cuda.stream(side):
        layer(x, out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer(x, out)
    for seed in (3, 4):
        x.copy_(synth.bf16_normal((80, 256), 1.0, seed=seed, device=DEV))
        want = layer(x).clone()
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert moeq.get_device_error() == 0
