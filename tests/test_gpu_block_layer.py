"""The norm, the scored router and the products with an epilogue as a layer runs
them: residual + norm (bf16 for the router, FP8 for a shared expert), routing by
biased sigmoid scores in groups, biased FP8 experts, the shared expert onto the
experts' sum, and the gradients of it all back to the layer's input.  Each step is
compared with its definition on the inputs that the step before gave."""
import numpy as np
import pytest
import torch

from fp4_fp8_quantization_gb300 import moeq, synth
from oracle import experts as X
from oracle import formats as F
from oracle import layers as L
from tests._util import DEV, assert_gemm_close, bf16_bits, need_gpu, u8
from tests.test_gpu_experts import EPS, U, close, f64

pytestmark = pytest.mark.gpu
BF16, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
T, E, K, G, SOME, H, I = 150, 32, 4, 8, 3, 512, 272
R = T * K


def _new(dtype, *shape):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def _blocks(n):
    return (n + 127) // 128


def _weight(e, n, k, seed):
    w = synth.bf16_normal((e, n, k), k ** -0.5, seed=seed, device=DEV)
    q, s = _new(U8, e, n, k), _new(F32, e, _blocks(n), _blocks(k))
    moeq.quantize_fp8_block_weight(w, q, s)
    return q, s


class Block:
    """Weights and workspaces of one layer; forward and backward only launch."""

    def __init__(self):
        self.norm_w = (1 + 0.1 * synth.bf16_normal((H,), 1.0, seed=1).float()).bfloat16().to(DEV)
        self.router = synth.bf16_normal((E, H), 0.05, seed=2, device=DEV)
        self.balance = synth.uniform((E,), -0.05, 0.05, seed=3, device=DEV)
        self.up, self.down = _weight(E, I, H, 4), _weight(E, H, I, 5)
        self.s_up, self.s_down = _weight(1, I, H, 6), _weight(1, H, I, 7)
        self.b_up, self.b_down = (synth.uniform((E, n), -0.5, 0.5, seed=8, device=DEV) for n in (I, H))
        self.all_rows = torch.tensor([0, T], dtype=I32, device=DEV)
        self.one = _new(I32, 1)
        n = self
        n.h, n.y, n.q, n.sq, n.rstd = (_new(BF16, T, H), _new(BF16, T, H), _new(U8, T, H),
                                       _new(F32, T, _blocks(H)), _new(F32, T))
        n.logits, n.ids, n.w = _new(BF16, T, E), _new(I32, T, K), _new(F32, T, K)
        n.ro, n.eids, n.src, n.dst = _new(I32, E + 1), _new(I32, E), _new(I32, R), _new(I32, T, K)
        n.a, n.sa = _new(U8, R, H), _new(F32, R, _blocks(H))
        n.z, n.u, n.qu, n.su = _new(BF16, R, I), _new(BF16, R, I), _new(U8, R, I), _new(F32, R, _blocks(I))
        n.rows, n.mixed, n.out = _new(BF16, R, H), _new(BF16, T, H), _new(BF16, T, H)
        n.su1, n.qs, n.ss = _new(BF16, T, I), _new(U8, T, I), _new(F32, T, _blocks(I))
        # gradients
        n.d_rows, n.d_w, n.d_logits = _new(BF16, R, H), _new(F32, T, K), _new(BF16, T, E)
        n.dq, n.dsq, n.db_down = _new(U8, R, H), _new(F32, R, _blocks(H)), _new(F32, E, H)
        n.d_u, n.dqz, n.dsz, n.db_up = _new(BF16, R, I), _new(U8, R, I), _new(F32, R, _blocks(I)), _new(F32, E, I)
        n.d_a, n.d_y, n.d_x, n.d_norm = _new(BF16, R, H), _new(BF16, T, H), _new(BF16, T, H), _new(F32, H)
        n.ws = [_new(U8, moeq.grouped_epilogue_grad_workspace(R, H, E)),
                _new(U8, moeq.add_rms_norm_grad_workspace(T, H))]
        t = lambda w: (w[0].transpose(1, 2).contiguous(), w[1].transpose(1, 2).contiguous())  # noqa: E731
        n.up_t, n.down_t = t(n.up), t(n.down)

    def forward(n, x, stream):
        moeq.add_rms_norm(x, n.norm_w, y=n.y, residual=stream, h=n.h, q=n.q, scales=n.sq, rstd=n.rstd)
        torch.mm(n.y, n.router.t(), out=n.logits)
        moeq.gate_group_topk(n.logits, n.ids, n.w, bias=n.balance, num_groups=G, topk_groups=SOME, scale=2.5)
        moeq.route_topk(n.ids, n.ro, n.eids, n.src, dst_info=n.dst)
        moeq.quantize_fp8_block_topk(n.y, n.dst, n.a, n.sa)
        moeq.grouped_matmul_fp8_block_epilogue(n.u, n.a, n.up[0], n.sa, n.up[1], n.ro, n.eids, bias=n.b_up,
                                               activation="gelu_tanh", z=n.z)
        moeq.quantize_fp8_block(n.u, n.qu, n.su)
        moeq.grouped_matmul_fp8_block_epilogue(n.rows, n.qu, n.down[0], n.su, n.down[1], n.ro, n.eids,
                                               bias=n.b_down)
        moeq.combine_topk(n.rows, n.dst, n.mixed, weights=n.w)
        moeq.grouped_matmul_fp8_block_epilogue(n.su1, n.q, n.s_up[0], n.sq, n.s_up[1], n.all_rows, n.one,
                                               activation="silu")
        moeq.quantize_fp8_block(n.su1, n.qs, n.ss)
        moeq.grouped_matmul_fp8_block_epilogue(n.out, n.qs, n.s_down[0], n.ss, n.s_down[1], n.all_rows, n.one,
                                               residual=n.mixed)

    def backward(n, d_out, d_h):
        """Through the routed experts, the router and the norm; d_h reaches the stream."""
        moeq.combine_topk_grad(d_out, n.dst, n.d_rows, weights=n.w, rows=n.rows, d_weights=n.d_w)
        moeq.grouped_epilogue_grad(n.d_rows, n.ro, n.eids, E, q=n.dq, scales=n.dsq, d_bias=n.db_down,
                                   workspace=n.ws[0])
        moeq.grouped_matmul_fp8_block(n.d_u, n.dq, n.down_t[0], n.dsq, n.down_t[1], n.ro, n.eids)
        moeq.grouped_epilogue_grad(n.d_u, n.ro, n.eids, E, z=n.z, activation="gelu_tanh", q=n.dqz,
                                   scales=n.dsz, d_bias=n.db_up, workspace=n.ws[0])
        moeq.grouped_matmul_fp8_block(n.d_a, n.dqz, n.up_t[0], n.dsz, n.up_t[1], n.ro, n.eids)
        moeq.permute_topk_grad(n.d_a, n.dst, n.d_y)
        moeq.gate_group_topk_grad(n.logits, n.ids, n.d_w, n.d_logits, scale=2.5)
        n.d_y.addmm_(n.d_logits, n.router)
        moeq.add_rms_norm_grad(n.d_y, n.h, n.norm_w, n.rstd, n.d_x, d_weight=n.d_norm, d_h=d_h,
                               workspace=n.ws[1])


def _inputs(seed):
    return tuple(synth.bf16_normal((T, H), s, seed=seed + i, device=DEV) for i, s in enumerate((1.0, 2.0, 0.1, 0.1)))


@pytest.fixture(scope="module")
def block():
    need_gpu()
    return Block()


def _product(z, want_z, c, act, residual=None):
    """z and c of a product against the reference of z."""
    if z is not None:
        assert_gemm_close(bf16_bits(z), want_z)
    want = L.epilogue(want_z, act, residual)
    ulp = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 1e-300))) - 7)
    assert np.all(np.abs(f64(c) - want) <= np.maximum(2 * ulp, 1.2e-3 * np.sqrt(np.mean(want_z ** 2))))


def test_layer_step_by_step(block):
    moeq.clear_device_error()
    n = block
    x, stream, d_out, d_h = _inputs(20)
    n.forward(x, stream)
    h = (x.float() + stream.float()).bfloat16()
    assert torch.equal(n.h, h)
    v, rstd = L.rms_norm(f64(h), f64(n.norm_w), 1e-6)
    close(n.y, v, (32 * EPS + U[BF16]) * np.abs(v))
    ids, w = L.gate_group_topk(f64(n.logits), K, f64(n.balance), groups=G, topk_groups=SOME, scale=2.5)
    assert np.array_equal(n.ids.cpu().numpy(), ids)
    close(n.w, w, 14 * EPS * w)
    ro, eids, dst = (t.cpu().numpy() for t in (n.ro, n.eids, n.dst))
    experts = L.row_experts(ro, eids, R)
    z = X.matmul(u8(n.a), u8(n.up[0]), f64(n.sa), f64(n.up[1]), ro, eids) + f64(n.b_up)[experts]
    _product(n.z, z, n.u, "gelu_tanh")
    z = X.matmul(u8(n.qu), u8(n.down[0]), f64(n.su), f64(n.down[1]), ro, eids) + f64(n.b_down)[experts]
    _product(None, z, n.rows, None)
    y, mag = X.collect(f64(n.rows), dst, f64(n.w))
    close(n.mixed, y, U[BF16] * np.abs(y) + 8 * EPS * mag)
    every, one = np.array([0, T]), np.array([0])
    _product(None, X.matmul(u8(n.q), u8(n.s_up[0]), f64(n.sq), f64(n.s_up[1]), every, one), n.su1, "silu")
    _product(None, X.matmul(u8(n.qs), u8(n.s_down[0]), f64(n.ss), f64(n.s_down[1]), every, one), n.out, None,
             f64(n.mixed))
    # back
    n.backward(d_out, d_h)
    _, ref, mag = L.epilogue_grad(f64(n.d_rows), None, None, experts, E)
    close(n.db_down, ref, (24 + R / 64 + 5) * EPS * mag + 1e-30)
    dz, ref, mag = L.epilogue_grad(f64(n.d_u), f64(n.z), "gelu_tanh", experts, E)
    slope = np.zeros((E, I))
    np.add.at(slope, experts, 1.5e-6 * np.abs(f64(n.d_u)))
    close(n.db_up, ref, (24 + R / 64 + 5) * EPS * mag + slope + 1e-30)
    got = F.decode_e4m3(u8(n.dqz)) * f64(n.dsz)[:, np.arange(I) // 128]
    assert np.all(np.abs(got - dz) <= 2.0 ** -4 * np.abs(dz) + 2.0 ** -10 * f64(n.dsz)[:, np.arange(I) // 128]
                  + 2e-6 * np.abs(f64(n.d_u)))
    ref = X.matmul(u8(n.dqz), u8(n.up_t[0]), f64(n.dsz), f64(n.up_t[1]), ro, eids)
    assert_gemm_close(bf16_bits(n.d_a), ref)
    ref = L.gate_group_topk_grad(f64(n.logits), ids, f64(n.d_w), "sigmoid", True, 2.5)
    size = 2.5 * np.abs(f64(n.d_w)).max(1, keepdims=True)
    close(n.d_logits, ref, 88 * EPS * size + U[BF16] * np.abs(ref))
    ref, ref_w, mag = L.rms_norm_grad(f64(h), f64(n.norm_w), 1e-6, f64(n.d_y), f64(d_h))
    g = np.abs(f64(n.d_y) * f64(n.norm_w))
    size = (g + np.abs(f64(h)) * rstd[:, None] ** 2 * (g * np.abs(f64(h))).mean(1, keepdims=True)) * rstd[:, None]
    close(n.d_x, ref, 96 * EPS * size + U[BF16] * np.abs(ref) + EPS * np.abs(f64(d_h)))
    close(n.d_norm, ref_w, (32 + 51) * EPS * mag + 1e-30)
    assert moeq.get_device_error() == 0


def test_layer_in_a_cuda_graph(block):
    """Forward and backward captured together give, replayed on other inputs, the bits of
    the direct calls, and allocate nothing."""
    moeq.clear_device_error()
    n = block
    ins = [t.clone() for t in _inputs(30)]
    run = lambda: (n.forward(ins[0], ins[1]), n.backward(ins[2], ins[3]))               # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    outs = (n.out, n.ids, n.w, n.d_x, n.d_norm, n.db_up, n.db_down, n.d_logits)
    for seed in (40, 50):
        for t, s in zip(ins, _inputs(seed)):
            t.copy_(s)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            run()
        side.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert moeq.get_device_error() == 0


class Norm(torch.autograd.Function):
    """x, residual, weight -> y, h"""

    @staticmethod
    def forward(ctx, x, res, w):
        y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(x.shape[0], device=x.device)
        moeq.add_rms_norm(x, w, y=y, residual=res, h=h, rstd=rstd, eps=1e-5)
        ctx.save_for_backward(h, w, rstd)
        return y, h

    @staticmethod
    def backward(ctx, d_y, d_h):
        h, w, rstd = ctx.saved_tensors
        d_x, d_w = torch.empty_like(h), torch.empty(h.shape[1], device=h.device)
        moeq.add_rms_norm_grad(d_y.contiguous(), h, w, rstd, d_x, d_weight=d_w, d_h=d_h.contiguous())
        return d_x, d_x, d_w.to(w.dtype)


class Gate(torch.autograd.Function):
    """logits -> weights of the experts chosen by biased scores in groups"""

    @staticmethod
    def forward(ctx, logits, bias, k):
        ids = torch.empty(logits.shape[0], k, dtype=I32, device=DEV)
        w = torch.empty(logits.shape[0], k, device=DEV)
        moeq.gate_group_topk(logits, ids, w, bias=bias, num_groups=4, topk_groups=2)
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    def backward(ctx, _, d_w):
        logits, ids = ctx.saved_tensors
        d = torch.empty_like(logits)
        moeq.gate_group_topk_grad(logits, ids, d_w.contiguous(), d)
        return d, None, None


def test_norm_and_router_as_autograd_functions():
    """Against autograd through the definitions, fp32: a dot product of 256 terms on both
    sides and the router's few, 2^-24 each."""
    need_gpu()
    g = torch.Generator(DEV).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)                            # noqa: E731
    x, res, w, router = rnd(40, 256), rnd(40, 256), 1 + 0.1 * rnd(256), rnd(16, 256) * 0.06
    bias, up, dh = 0.05 * rnd(16), rnd(40, 4), rnd(40, 256)

    def ours(x, res, w, router):
        y, h = Norm.apply(x, res, w)
        ids, p = Gate.apply(y @ router.t(), bias, 4)
        return (p * up).sum() + (h * dh).sum(), ids

    def plain(x, res, w, router):
        h = x + res
        y = h * (h.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w
        s = torch.sigmoid(y @ router.t())
        c = s.detach() + bias
        value = c.view(-1, 4, 4).topk(2, dim=2).values.sum(2)
        keep = torch.zeros_like(value, dtype=torch.bool).scatter(1, value.topk(2, dim=1).indices, True)
        ids = c.masked_fill(~keep.repeat_interleave(4, 1), -9.0).topk(4, dim=1).indices
        p = s.gather(1, ids)
        return (p / p.sum(1, keepdim=True) * up).sum() + (h * dh).sum(), ids

    grads = []
    for f in (ours, plain):
        leaves = [t.clone().requires_grad_() for t in (x, res, w, router)]
        loss, ids = f(*leaves)
        loss.backward()
        grads.append(([t.grad for t in leaves], ids.long()))
    assert torch.equal(grads[0][1], grads[1][1])
    for a, b in zip(*(v[0] for v in grads)):
        assert float((a - b).norm() / b.norm()) < 1e-5
    assert moeq.get_device_error() == 0
