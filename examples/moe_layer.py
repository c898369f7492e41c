"""A mixture-of-experts layer on the library's calls, serving and training.

``python examples/moe_layer.py`` runs both on cuda:0 with random weights:

* serving: router, routing, tokens quantized into their experts' rows, gate/up
  product, SwiGLU requantized, down product and the way back, all in FP8 with
  128-block scales;
* training: the router's and the rows' gradients as autograd functions around
  experts in plain bf16 PyTorch, a few steps that fit a teacher layer.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp4_fp8_quantization_gb300 import moeq  # noqa: E402

F8 = torch.float8_e4m3fn


def _i32(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def _blocks(n):
    return (n + 127) // 128


class Fp8MoeLayer:
    """y = sum over a token's top_k experts of w * down(swiglu(gate_up(x))).

    router bf16 [E, H]; gate_up bf16 [E, 2 I, H] with row 2 j = gate_j, 2 j + 1 =
    up_j; down bf16 [E, H, I].  Weights are quantized once; workspaces for up to
    max_tokens tokens are kept, so that a call given its output allocates nothing
    (and can be captured in a CUDA graph)."""

    def __init__(self, router, gate_up, down, top_k, max_tokens):
        self.E, two_i, self.H = gate_up.shape
        self.I, self.k, self.router = two_i // 2, top_k, router
        self.w1, self.s1 = self._weight(gate_up)
        self.w2, self.s2 = self._weight(down)
        T, R = max_tokens, max_tokens * top_k
        new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.logits = new(T, self.E, dtype=router.dtype)
        self.ids, self.weights, self.dst = _i32(T, top_k), new(T, top_k), _i32(T, top_k)
        self.offsets, self.experts, self.src = _i32(self.E + 1), _i32(self.E), _i32(R)
        self.a, self.sa = new(R, self.H, dtype=F8), new(R, _blocks(self.H))
        self.y = new(R, two_i, dtype=torch.bfloat16)
        self.h, self.sh = new(R, self.I, dtype=F8), new(R, _blocks(self.I))
        self.z = new(R, self.H, dtype=torch.bfloat16)

    @staticmethod
    def _weight(w):
        E, N, K = w.shape
        q = torch.empty(w.shape, dtype=F8, device="cuda")
        s = torch.empty((E, _blocks(N), _blocks(K)), device="cuda")
        moeq.quantize_fp8_block_weight(w, q, s)
        return q, s

    @torch.no_grad()
    def __call__(self, x, out=None):
        T, R = x.shape[0], x.shape[0] * self.k
        out = torch.empty_like(x) if out is None else out
        ids, w, dst = self.ids[:T], self.weights[:T], self.dst[:T]
        logits = torch.mm(x, self.router.t(), out=self.logits[:T])
        moeq.gate_topk(logits, ids, w)
        moeq.route_topk(ids, self.offsets, self.experts, self.src, dst_info=dst)
        moeq.quantize_fp8_block_topk(x, dst, self.a[:R], self.sa[:R])
        moeq.grouped_matmul_fp8_block(self.y[:R], self.a[:R], self.w1, self.sa[:R], self.s1,
                                      self.offsets, self.experts)
        moeq.swiglu_quantize_fp8_block(self.y[:R], self.h[:R], self.sh[:R])
        moeq.grouped_matmul_fp8_block(self.z[:R], self.h[:R], self.w2, self.sh[:R], self.s2,
                                      self.offsets, self.experts)
        moeq.combine_topk(self.z[:R], dst, out, weights=w)
        return out


class Router(torch.autograd.Function):
    """logits -> (ids, weights)"""

    @staticmethod
    def forward(ctx, logits, top_k):
        T = logits.shape[0]
        ids, w = _i32(T, top_k), torch.empty(T, top_k, device="cuda")
        moeq.gate_topk(logits, ids, w)
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    def backward(ctx, _, d_w):
        logits, ids = ctx.saved_tensors
        d_logits = torch.empty_like(logits, memory_format=torch.contiguous_format)
        moeq.gate_topk_grad(logits, ids, d_w.contiguous(), d_logits)
        return d_logits, None


class Permute(torch.autograd.Function):
    """tokens -> their experts' rows"""

    @staticmethod
    def forward(ctx, x, dst):
        rows = torch.zeros(dst.numel(), x.shape[1], dtype=x.dtype, device="cuda")
        moeq.permute_topk(x, dst, rows)
        ctx.save_for_backward(dst)
        return rows

    @staticmethod
    def backward(ctx, d_rows):
        dst, = ctx.saved_tensors
        d_x = torch.empty(dst.shape[0], d_rows.shape[1], dtype=d_rows.dtype, device="cuda")
        moeq.permute_topk_grad(d_rows.contiguous(), dst, d_x)
        return d_x, None


class Combine(torch.autograd.Function):
    """rows, weights -> tokens"""

    @staticmethod
    def forward(ctx, rows, w, dst):
        out = torch.empty(dst.shape[0], rows.shape[1], dtype=rows.dtype, device="cuda")
        moeq.combine_topk(rows, dst, out, weights=w)
        ctx.save_for_backward(rows, w, dst)
        return out

    @staticmethod
    def backward(ctx, d_out):
        rows, w, dst = ctx.saved_tensors
        d_rows, d_w = torch.zeros_like(rows), torch.empty_like(w)
        moeq.combine_topk_grad(d_out.contiguous(), dst, d_rows, weights=w, rows=rows, d_weights=d_w)
        return d_rows, d_w, None


def route(ids, num_experts):
    """(row of each choice, row offsets on the host)"""
    dst, offsets = _i32(*ids.shape), _i32(num_experts + 1)
    moeq.route_topk(ids, offsets, _i32(num_experts), _i32(ids.numel()), dst_info=dst)
    return dst, offsets.tolist()


def trained_layer(x, router, gate_up, down, top_k):
    """The same layer for training: bf16 experts, one after another."""
    ids, w = Router.apply(x.float() @ router.float().t(), top_k)
    dst, off = route(ids, gate_up.shape[0])
    rows = Permute.apply(x, dst)
    parts = []
    for e in range(gate_up.shape[0]):
        y = rows[off[e]:off[e + 1]] @ gate_up[e].t()
        parts.append((torch.nn.functional.silu(y[:, 0::2]) * y[:, 1::2]) @ down[e].t())
    return Combine.apply(torch.cat(parts), w, dst)


def plain_layer(x, router, gate_up, down, top_k):
    """The definition in fp32, every expert on every token."""
    logits = x.float() @ router.float().t()
    val, ids = logits.topk(top_k, dim=1)
    w = torch.zeros_like(logits).scatter(1, ids, torch.softmax(val, 1))
    y = torch.einsum("th,enh->ten", x.float(), gate_up.float())
    h = torch.nn.functional.silu(y[..., 0::2]) * y[..., 1::2]
    return torch.einsum("te,tei,ehi->th", w, h, down.float())


def make_weights(E, H, I, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).bfloat16()  # noqa: E731
    return rnd(E, H) * 4, rnd(E, 2 * I, H), rnd(E, H, I)


def serve(T=512, E=16, H=1024, I=384, top_k=4):
    """Relative error of the FP8 layer against the definition."""
    weights = make_weights(E, H, I, seed=1)
    x = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    layer = Fp8MoeLayer(*weights, top_k=top_k, max_tokens=T)
    out = layer(x).float()
    one = layer(x[:1]).float()          # a single token through the same workspaces
    ref = plain_layer(x, *weights, top_k)
    assert moeq.get_device_error() == 0
    return float((out - ref).norm() / ref.norm()), float((one - ref[:1]).norm() / ref[:1].norm())


def train(T=256, E=8, H=256, I=128, top_k=2, steps=30):
    """Loss before and after some steps towards a teacher layer."""
    teacher = make_weights(E, H, I, seed=3)
    params = [w.float().requires_grad_() for w in make_weights(E, H, I, seed=4)]
    x = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(5)).bfloat16()
    want = plain_layer(x, *teacher, top_k)
    opt = torch.optim.Adam(params, lr=3e-3)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = (trained_layer(x, *(p.bfloat16() for p in params), top_k).float() - want).square().mean()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    assert moeq.get_device_error() == 0
    return losses[0], losses[-1]


if __name__ == "__main__":
    print("serving: relative error %.4f (512 tokens), %.4f (one token)" % serve())
    print("training: loss %.4f -> %.4f" % train())
