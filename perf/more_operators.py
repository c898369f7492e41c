"""What stands around a mixture-of-experts layer's products: the residual's
addition with the root-mean-square norm and its 8-bit output, the router that
scores experts with a balance bias and groups, and the grouped FP8 product with
bias, activation and residual in its epilogue, with their gradients.

``run`` computes them with plain tensor operations in 32 bits (a router's choice
in 64), or, where ``own`` is true, by the calls of
``fp4_fp8_quantization_gb300.moeq``; ``exact`` computes them from their
definitions in 64 bits.  A case is a dict:

``op``      gate | norm | matmul
``pass``    forward | training (forward and gradient), for gate and norm;
            forward | saving (the pre-activation is stored too) | gradient (of
            the epilogue, from the stored pre-activation), for matmul
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the router of one decode batch: sigmoid scores, a balance bias, 4 of 8 groups
        dict(name="gate decode", op="gate", tokens=64, experts=256, groups=8, topk_groups=4,
             top_k=8, score="sigmoid", bias=True, group_score="top2", normalize=True, scale=2.5,
             dtype="bf16", masked=False, **{"pass": "forward"}),
        # the same router in a training step, logits kept in fp32
        dict(name="gate training", op="gate", tokens=65537, experts=256, groups=8, topk_groups=4,
             top_k=8, score="sigmoid", bias=True, group_score="top2", normalize=True, scale=2.5,
             dtype="fp32", masked=False, **{"pass": "training"}),
        # softmax scores, groups by their best expert, group sizes that are no power of two
        dict(name="gate softmax groups", op="gate", tokens=9999, experts=160, groups=8,
             topk_groups=3, top_k=6, score="softmax", bias=False, group_score="max",
             normalize=False, scale=16.0, dtype="bf16", masked=False, **{"pass": "forward"}),
        # before a decode batch's router and shared expert: y for the one, codes for the other
        dict(name="norm decode", op="norm", rows=16, cols=7168, dtype="bf16", residual=True,
             y=True, codes="block", **{"pass": "forward"}),
        # a prompt of an odd length, codes for the next product only
        dict(name="norm prompt", op="norm", rows=8191, cols=4096, dtype="bf16", residual=True,
             y=False, codes="block", **{"pass": "forward"}),
        # a training step's norm and its gradient
        dict(name="norm training", op="norm", rows=16384, cols=7168, dtype="bf16", residual=True,
             y=True, codes="none", **{"pass": "training"}),
        # fp16, no residual, codes with one scale per row, rows that fill no power of two
        dict(name="norm rows training", op="norm", rows=5003, cols=2480, dtype="fp16",
             residual=False, y=True, codes="row", **{"pass": "training"}),
        # one token's eight experts with biases, gate/up side
        dict(name="product one token", op="matmul", tokens=1, top_k=8, experts=128, k=4096, n=1536,
             zipf=0.0, bias=True, act="silu", residual=False, **{"pass": "forward"}),
        # a dense layer's output product for one decode batch, onto the residual stream
        dict(name="product decode", op="matmul", tokens=64, top_k=1, experts=1, k=4096, n=4096,
             zipf=0.0, bias=True, act="none", residual=True, **{"pass": "forward"}),
        # a skewed prompt on sizes that end inside a block and inside a tile, in training
        dict(name="product ragged", op="matmul", tokens=2999, top_k=4, experts=48, k=2480, n=1904,
             zipf=0.6, bias=True, act="gelu", residual=False, **{"pass": "saving"}),
        # a dense layer over a large prompt
        dict(name="product prompt", op="matmul", tokens=16384, top_k=1, experts=1, k=4096, n=7168,
             zipf=0.0, bias=True, act="gelu_tanh", residual=True, **{"pass": "forward"}),
        # the epilogue's gradient of a training step: 32768 rows over 64 experts
        dict(name="epilogue gradient", op="matmul", tokens=4096, top_k=8, experts=64, k=4096,
             n=4096, zipf=0.3, bias=True, act="silu", residual=False, **{"pass": "gradient"}),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi + 0.999)))) - 0.4))))


def draw(rng):
    op = rng.choice(["gate", "norm", "matmul", "matmul"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 3, 4, 8, 16])
        size = _log(rng, max(4, 8 // groups), 512 // groups)
        some, e = rng.randint(1, groups), groups * size
        return dict(op=op, tokens=_log(rng, 1, 16 * 1024 * 1024 // e), experts=e, groups=groups,
                    topk_groups=some, top_k=rng.randint(1, min(8, some * size)),
                    score=rng.choice(["sigmoid", "sigmoid", "softmax"]), bias=rng.random() < 0.7,
                    group_score=rng.choice(["top2", "max"]), normalize=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    masked=rng.random() < 0.3, **{"pass": rng.choice(["forward", "training"])})
    if op == "norm":
        cols = 16 * _log(rng, 4, 512)
        codes = rng.choice(["none", "block", "block", "row"])
        return dict(op=op, rows=_log(rng, 1, min(65536, 110_000_000 // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), residual=rng.random() < 0.7,
                    y=codes == "none" or rng.random() < 0.5, codes=codes,
                    **{"pass": rng.choice(["forward", "training"])})
    k, n, e = 16 * _log(rng, 8, 448), 16 * _log(rng, 8, 448), _log(rng, 1, 128)
    top_k = rng.randint(1, min(8, e))
    most = min(65536, 16384 * 4096 * 7168 // (k * n)) // top_k
    return dict(op=op, tokens=_log(rng, 1, max(1, most)), top_k=top_k, experts=e, k=k, n=n,
                zipf=rng.choice([0.0, 0.0, 0.5]), bias=rng.random() < 0.7,
                act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                residual=rng.random() < 0.5,
                **{"pass": rng.choice(["forward", "forward", "saving", "gradient"])})


def _blocks(n):
    return -(-n // BLOCK)


def _size(case):
    return 4 if case["dtype"] == "fp32" else 2


def work(case):
    op = case["op"]
    if op == "gate":
        t, e, k, size = case["tokens"], case["experts"], case["top_k"], _size(case)
        b, f = t * e * size + 4 * e * case["bias"] + 8 * t * k, 5 * t * e
        if case["pass"] == "training":
            # the choice is fixed: the gradient needs the chosen logits, or, for a softmax
            # over all, every one; it writes the whole rows
            read = e if case["score"] == "softmax" and not case["normalize"] else k
            b, f = b + t * (read + e) * size + 8 * t * k, f + 8 * t * read
        return {"bytes": b, "flops": f}
    if op == "norm":
        n, r, size = case["rows"] * case["cols"], case["rows"], _size(case)
        b = n * size * (1 + 2 * case["residual"] + case["y"]) + size * case["cols"]
        if case["codes"] != "none":
            b += n + 4 * r * (_blocks(case["cols"]) if case["codes"] == "block" else 1)
        f = 6 * n
        if case["pass"] == "training":
            b += n * size * (3 + case["residual"]) + (size + 4) * case["cols"] + 8 * r
            f += 10 * n
        return {"bytes": b, "flops": f}
    rows, k, n, e = case["tokens"] * case["top_k"], case["k"], case["n"], case["experts"]
    if case["pass"] == "gradient":
        b = rows * n * (2 + 2 * (case["act"] != "none") + 1) + 4 * rows * _blocks(n)
        return {"bytes": b + 4 * e * n * case["bias"], "flops": 12 * rows * n}
    # experts with rows, as many as even routing is expected to reach
    active = e * (1.0 - (1.0 - min(1.0, case["top_k"] / e)) ** case["tokens"])
    out = 2 * n * (1 + case["residual"] + (case["pass"] == "saving"))
    b = (rows * (k + 4 * _blocks(k) + out)
         + max(1, int(active)) * (n * k + 4 * _blocks(n) * _blocks(k) + 4 * n * case["bias"]) + 8 * e)
    return {"bytes": b, "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _counts(tokens, experts, top_k, g, zipf):
    """Rows of each expert when every token takes top_k different ones."""
    p = -zipf * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    u = torch.rand(tokens, experts, generator=g, device="cuda").clamp_(1e-12, 1.0 - 1e-7)
    ids = (p - torch.log(-torch.log(u))).topk(top_k, dim=1).indices.reshape(-1)
    return torch.bincount(ids, minlength=experts)


def _activations(g, rows, cols):
    """N(0, 1) with one element in a hundred ten times as large."""
    x = _rand(g, rows, cols)
    return x.mul_(1.0 + 9.0 * (torch.rand(rows, cols, generator=g, device="cuda") < 0.01))


def _prepare_gate(s, g):
    t, e, k, dt = s["tokens"], s["experts"], s["top_k"], DTYPES[s["dtype"]]
    x = _rand(g, t, e) * 1.5
    if s["masked"]:
        # experts that a token may not use: a run of an eighth of them, the start differing
        at = torch.randint(0, e, (t, 1), generator=g, device="cuda")
        x = x.masked_fill((torch.arange(e, device="cuda") - at) % e < e // 8, float("-inf"))
    s["logits"] = x.to(dt)
    # a bias of about the spread of the scores that compete
    s["b"] = _rand(g, e) * (0.05 if s["score"] == "sigmoid" else 0.5 / e) if s["bias"] else None
    s["ids"] = torch.empty(t, k, dtype=torch.int32, device="cuda")
    s["weights"] = torch.empty(t, k, device="cuda")
    if s["pass"] == "training":
        s["d_weights"] = _rand(g, t, k)
        s["d_logits"] = torch.empty_like(s["logits"])


def _prepare_norm(s, g):
    r, c, dt = s["rows"], s["cols"], DTYPES[s["dtype"]]
    s["x"] = _activations(g, r, c).to(dt)
    s["res"] = (_activations(g, r, c) * 2.0).to(dt) if s["residual"] else None
    s["w"] = (1.0 + 0.2 * _rand(g, c)).to(dt)
    empty = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    s["h"] = empty(r, c, dtype=dt) if s["residual"] else None
    s["out"] = empty(r, c, dtype=dt) if s["y"] else None
    s["q"] = s["sf"] = s["rstd"] = None
    if s["codes"] != "none":
        s["q"] = empty(r, c, dtype=torch.float8_e4m3fn)
        s["sf"] = empty(r, _blocks(c)) if s["codes"] == "block" else empty(r)
    if s["pass"] == "training":
        s["rstd"], s["dx"], s["dw"] = empty(r), empty(r, c, dtype=dt), empty(c)
        s["dy"] = _rand(g, r, c).to(dt)
        s["dh"] = _rand(g, r, c).to(dt) if s["residual"] else None


def _prepare_matmul(s, g):
    t, k, n, e = s["tokens"] * s["top_k"], s["k"], s["n"], s["experts"]
    counts = _counts(s["tokens"], e, s["top_k"], g, s["zipf"])
    s["offsets"] = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    s["offsets"][1:] = counts.cumsum(0)
    s["ids"] = torch.arange(e, dtype=torch.int32, device="cuda")
    s["most"], s["active"] = int(counts.max()), int((counts > 0).sum())
    if s["pass"] == "gradient":
        s["dc"] = (_rand(g, t, n) * 0.01).to(torch.bfloat16)
        s["z"] = (_rand(g, t, n) * 1.5).to(torch.bfloat16) if s["act"] != "none" else None
        s["q"] = torch.empty(t, n, dtype=torch.float8_e4m3fn, device="cuda")
        s["sf"] = torch.empty(t, _blocks(n), device="cuda")
        s["db"] = torch.empty(e, n, device="cuda") if s["bias"] else None
        return
    s["a"], s["sa"] = _quantize_rows(_activations(g, t, k).to(torch.bfloat16).float())
    # weights as they are loaded: quantized once, a few experts at a time
    s["b"] = torch.empty(e, n, k, dtype=torch.float8_e4m3fn, device="cuda")
    s["sb"] = torch.empty(e, _blocks(n), _blocks(k), device="cuda")
    step = max(1, 200_000_000 // (n * k))
    for i in range(0, e, step):
        m = min(step, e - i)
        s["b"][i:i + m], s["sb"][i:i + m] = _quantize_weight(_rand(g, m, n, k) * k ** -0.5)
    s["bias_v"] = _rand(g, e, n) * 0.5 if s["bias"] else None
    s["res"] = (_rand(g, t, n) * 2.0).to(torch.bfloat16) if s["residual"] else None
    s["c"] = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    s["z"] = torch.empty_like(s["c"]) if s["pass"] == "saving" else None


def prepare(case, seed):
    g, s = _gen(seed), dict(case)
    {"gate": _prepare_gate, "norm": _prepare_norm, "matmul": _prepare_matmul}[s["op"]](s, g)
    return s


# ------------------------------------------- plain forms (32 bits, torch)

def _pad(x, *multiples):
    """x with its last len(multiples) axes padded by zeros to the multiples."""
    sizes = []
    for n, m in zip(reversed(x.shape[-len(multiples):]), reversed(multiples)):
        sizes += [0, -n % m]
    return torch.nn.functional.pad(x, sizes) if any(sizes) else x


def _codes(x, amax):
    """(E4M3 codes of x, scales) with one scale for each amax, keepdim shapes."""
    s = (amax / torch.full_like(amax, E4M3_MAX)).clamp_min(SCALE_MIN)
    q = (x * torch.reciprocal(s)).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn), s


def _quantize_rows(x):
    n, k = x.shape
    b = _pad(x, BLOCK).view(n, _blocks(k), BLOCK)
    q, s = _codes(b, b.abs().amax(-1, keepdim=True))
    return q.view(n, -1)[:, :k].contiguous(), s.view(n, -1)


def _quantize_weight(w):
    e, n, k = w.shape
    b = _pad(w, BLOCK, BLOCK).view(e, _blocks(n), BLOCK, _blocks(k), BLOCK)
    q, s = _codes(b, b.abs().amax((2, 4), keepdim=True))
    return (q.view(e, _blocks(n) * BLOCK, -1)[:, :n, :k].contiguous(),
            s.view(e, _blocks(n), _blocks(k)))


def _choose(s):
    """The choice, in 64 bits: scores next to one another decide it.  int64
    [tokens, top_k], -1 where a token has no expert left."""
    x, g = s["logits"].double(), s["groups"]
    score = 1.0 / (1.0 + torch.exp(-x)) if s["score"] == "sigmoid" else _softmax(x)
    off = x == float("-inf")
    # without a bias the order is that of the logits
    c = (x if s["b"] is None else score + s["b"].double()).masked_fill(off, float("-inf"))
    if g > 1:
        v = c if s["b"] is not None or s["group_score"] == "max" else score.masked_fill(off, float("-inf"))
        best = torch.sort(v.view(-1, g, v.shape[1] // g), dim=2, descending=True).values
        value = best[:, :, 0]
        if s["group_score"] == "top2" and best.shape[2] > 1:
            # a group with one usable expert counts that one
            value = torch.where(best[:, :, 1] > float("-inf"), value + best[:, :, 1], value)
        order = torch.sort(value, dim=1, descending=True, stable=True).indices
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order[:, :s["topk_groups"]], True)
        c = c.masked_fill(~keep.repeat_interleave(v.shape[1] // g, 1), float("-inf"))
    top = torch.sort(c, dim=1, descending=True, stable=True)
    k = s["top_k"]
    return top.indices[:, :k].masked_fill(top.values[:, :k] == float("-inf"), -1)


def _softmax(x):
    p = torch.exp(x - x.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _plain_gate(s):
    x, ids = s["logits"].float(), _choose(s)
    none, at = ids < 0, ids.clamp_min(0)
    p = torch.sigmoid(x) if s["score"] == "sigmoid" else _softmax(x)
    chosen = p.gather(1, at).masked_fill(none, 0.0)
    total = chosen.sum(1, keepdim=True) if s["normalize"] else torch.ones_like(chosen[:, :1])
    out = [ids.to(torch.int32), torch.where(total > 0, chosen / total * s["scale"], 0.0)]
    if s["pass"] == "training":
        d = s["d_weights"].masked_fill(none, 0.0) * s["scale"]
        if s["normalize"]:
            d = (d - (chosen / total * d).sum(1, keepdim=True)) / total
        # d is now the scores' gradient at the choices
        if s["score"] == "sigmoid":
            d = d * chosen * (1.0 - chosen)
            dx = torch.zeros_like(x).scatter_add(1, at, d.masked_fill(none, 0.0))
        elif s["normalize"]:
            # the softmax's own denominator cancels
            dx = torch.zeros_like(x).scatter_add(1, at, (d * chosen).masked_fill(none, 0.0))
        else:
            dp = torch.zeros_like(x).scatter_add(1, at, d.masked_fill(none, 0.0))
            dx = p * (dp - (chosen * d).sum(1, keepdim=True))
        out.append(dx.to(s["logits"].dtype))
    return out


def _plain_norm(s):
    dt = s["x"].dtype
    h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(dt)
    hf, w = h.float(), s["w"].float()
    rstd = torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS)
    y = hf * rstd * w
    out = {}
    if s["res"] is not None:
        out["h"] = h
    if s["y"]:
        out["y"] = y.to(dt)
    if s["codes"] == "block":
        out["q"], out["scales"] = _quantize_rows(y)
    elif s["codes"] == "row":
        q, sf = _codes(y, y.abs().amax(1, keepdim=True))
        out["q"], out["scales"] = q, sf.view(-1)
    if s["pass"] == "training":
        dy = s["dy"].float()
        wd = w * dy
        dx = rstd * (wd - hf * (rstd * rstd * (wd * hf).mean(1, keepdim=True)))
        out["d_x"] = (dx if s["dh"] is None else dx + s["dh"].float()).to(dt)
        out["d_weight"] = (dy * hf * rstd).sum(0)
        out["rstd"] = rstd.view(-1)
    return out


def _act(z, name):
    if name == "relu":
        return z.clamp_min(0.0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * np.pi) ** -0.5
    if name == "gelu_tanh":
        a = (2.0 / np.pi) ** 0.5
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _row_experts(s, rows):
    return torch.bucketize(torch.arange(rows, device="cuda"), s["offsets"].long()[1:], right=True)


def _plain_matmul(s):
    n, e = s["n"], s["active"]
    if s["pass"] == "gradient":
        dz = s["dc"].float()
        if s["z"] is not None:
            dz = dz * _act_slope(s["z"].float(), s["act"])
        q, sf = _quantize_rows(dz)
        out = {"q": q, "scales": sf}
        if s["bias"]:
            out["d_bias"] = torch.zeros(s["experts"], n, device="cuda").index_add_(
                0, _row_experts(s, dz.shape[0]), dz)
        return out
    # the rows of every expert that has some padded to the largest group, one batched product
    a = s["a"]
    offs, row = s["offsets"].long(), torch.arange(a.shape[0], device="cuda")
    live = torch.sort((offs.diff() > 0).int(), descending=True, stable=True).indices[:e]
    group = torch.bucketize(row, offs[1:][live], right=True)
    slot = group * s["most"] + row - offs[:-1][live][group]
    af = (_pad(a.float(), BLOCK).view(a.shape[0], -1, BLOCK) * s["sa"][:, :, None]).view(a.shape[0], -1)
    padded = torch.zeros(e * s["most"], af.shape[1], device="cuda")
    padded[slot] = af
    b = _pad(s["b"][live].float(), BLOCK, BLOCK).view(e, _blocks(n), BLOCK, -1, BLOCK)
    b = b.mul_(s["sb"][live][:, :, None, :, None]).view(e, _blocks(n) * BLOCK, -1)
    z = torch.bmm(padded.view(e, s["most"], -1), b.transpose(1, 2)).view(e * s["most"], -1)[slot, :n]
    if s["bias_v"] is not None:
        z = z + s["bias_v"][live][group]
    c = _act(z, s["act"])
    out = {"c": (c if s["res"] is None else c + s["res"].float()).to(torch.bfloat16)}
    if s["pass"] == "saving":
        out["z"] = z.to(torch.bfloat16)
    return out


# -------------------------------------------------- the framework's calls

def _own(s):
    from fp4_fp8_quantization_gb300 import moeq

    if s["op"] == "gate":
        moeq.gate_group_topk(s["logits"], s["ids"], s["weights"], bias=s["b"], score=s["score"],
                             num_groups=s["groups"], topk_groups=s["topk_groups"],
                             group_score=s["group_score"], normalize=s["normalize"],
                             scale=s["scale"])
        if s["pass"] == "forward":
            return [s["ids"], s["weights"]]
        moeq.gate_group_topk_grad(s["logits"], s["ids"], s["d_weights"], s["d_logits"],
                                  score=s["score"], normalize=s["normalize"], scale=s["scale"])
        return [s["ids"], s["weights"], s["d_logits"]]
    if s["op"] == "norm":
        moeq.add_rms_norm(s["x"], s["w"], y=s["out"], residual=s["res"], h=s["h"], q=s["q"],
                          scales=s["sf"], rstd=s["rstd"], eps=EPS)
        out = {"h": s["h"], "y": s["out"], "q": s["q"], "scales": s["sf"]}
        if s["pass"] == "training":
            moeq.add_rms_norm_grad(s["dy"], s["x"] if s["h"] is None else s["h"], s["w"],
                                   s["rstd"], s["dx"], d_weight=s["dw"], d_h=s["dh"])
            out.update(d_x=s["dx"], d_weight=s["dw"], rstd=s["rstd"])
        return {k: v for k, v in out.items() if v is not None}
    act = None if s["act"] == "none" else s["act"]
    if s["pass"] == "gradient":
        moeq.grouped_epilogue_grad(s["dc"], s["offsets"], s["ids"], s["experts"], z=s["z"],
                                   activation=act, q=s["q"], scales=s["sf"], d_bias=s["db"])
        out = {"q": s["q"], "scales": s["sf"]}
        return {**out, "d_bias": s["db"]} if s["bias"] else out
    moeq.grouped_matmul_fp8_block_epilogue(
        s["c"], s["a"], s["b"], s["sa"], s["sb"], s["offsets"], s["ids"], bias=s["bias_v"],
        activation=act, residual=s["res"], z=s["z"], max_tokens_per_expert=s["most"])
    return {"c": s["c"], "z": s["z"]} if s["pass"] == "saving" else {"c": s["c"]}


def run(state):
    if own:
        return _own(state)
    return {"gate": _plain_gate, "norm": _plain_norm, "matmul": _plain_matmul}[state["op"]](state)


# ------------------------------------------- the definitions in 64 bits

def _e4m3_64(v):
    """The E4M3 value nearest to v (ties to the even code, saturating)."""
    mag = v.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(mag.clamp_min(2.0 ** -6))) - 3.0)
    return torch.copysign(torch.round(mag / step) * step, v)


def _exact_codes(x, width):
    """Codes' values and scales, one for each `width` columns (all: a flat list)."""
    part = torch.arange(x.shape[1], device="cuda") // width
    amax = torch.zeros(x.shape[0], int(part[-1]) + 1, dtype=torch.float64, device="cuda")
    amax = amax.scatter_reduce(1, part.expand_as(x), x.abs(), "amax")
    sf = (amax / E4M3_MAX).clamp_min(SCALE_MIN)
    return _e4m3_64(x / sf[:, part]), sf


def _exact_gate(s):
    x, ids = s["logits"].double(), _choose(s)
    none, at = ids < 0, ids.clamp_min(0)
    # logarithms of the scores
    log_p = (torch.nn.functional.logsigmoid(x) if s["score"] == "sigmoid"
             else x - torch.logsumexp(x, 1, keepdim=True))
    v = log_p.gather(1, at).masked_fill(none, float("-inf"))
    if s["normalize"]:
        v = v - torch.logsumexp(v, 1, keepdim=True)
    w = torch.exp(v).masked_fill(none, 0.0) * s["scale"]
    out = [None, w]
    if s["pass"] == "training":
        g = w * s["d_weights"].double()        # the gradient by log w
        if s["normalize"]:
            g = g - w / s["scale"] * g.sum(1, keepdim=True)
        # d log sigmoid = 1 - sigmoid; d log softmax_i / d x_j = [i = j] - p_j
        if s["score"] == "sigmoid":
            g = g * torch.sigmoid(-x).gather(1, at)
        dx = torch.zeros_like(x).scatter_add(1, at, g.masked_fill(none, 0.0))
        if s["score"] == "softmax" and not s["normalize"]:
            dx = dx - torch.exp(log_p) * g.sum(1, keepdim=True)
        out.append(dx)
    return out


def _exact_norm(s):
    dt = s["x"].dtype
    h = s["x"].double() if s["res"] is None else (s["x"].double() + s["res"].double()).to(dt).double()
    w, n = s["w"].double(), s["cols"]
    rstd = (torch.einsum("rc,rc->r", h, h) / n + EPS) ** -0.5
    y = torch.einsum("rc,r,c->rc", h, rstd, w)
    out = {}
    if s["res"] is not None:
        out["h"] = h
    if s["y"]:
        out["y"] = y
    if s["codes"] != "none":
        out["q"], sf = _exact_codes(y, BLOCK if s["codes"] == "block" else n)
        out["scales"] = sf if s["codes"] == "block" else sf.view(-1)
    if s["pass"] == "training":
        dy, unit = s["dy"].double(), h * rstd[:, None]
        d_unit = dy * w
        dx = (d_unit - unit * (torch.einsum("rc,rc->r", d_unit, unit) / n)[:, None]) * rstd[:, None]
        out["d_x"] = dx if s["dh"] is None else dx + s["dh"].double()
        out["d_weight"] = torch.einsum("rc,rc->c", dy, unit)
        out["rstd"] = rstd
    return out


def _act64(z, name):
    """(activation, its slope) by autograd through its definition."""
    z = z.detach().requires_grad_()
    with torch.enable_grad():
        f = torch.nn.functional
        c = {"none": lambda: z * 1.0, "relu": lambda: f.relu(z), "silu": lambda: f.silu(z),
             "gelu": lambda: f.gelu(z), "gelu_tanh": lambda: f.gelu(z, approximate="tanh")}[name]()
        slope, = torch.autograd.grad(c.sum(), z)
    return c.detach(), slope


def _exact_matmul(s):
    k, n = s["k"], s["n"]
    offs = s["offsets"].tolist()
    if s["pass"] == "gradient":
        dz = s["dc"].double()
        if s["z"] is not None:
            dz = dz * _act64(s["z"].double(), s["act"])[1]
        q, sf = _exact_codes(dz, BLOCK)
        out = {"q": q, "scales": sf}
        if s["bias"]:
            out["d_bias"] = torch.stack([dz[a:b].sum(0) for a, b in zip(offs, offs[1:])])
        return out
    kk, nn = torch.arange(k, device="cuda") // BLOCK, torch.arange(n, device="cuda") // BLOCK
    z = torch.empty(offs[-1], n, dtype=torch.float64, device="cuda")
    for e in range(len(offs) - 1):
        r0, r1 = offs[e], offs[e + 1]
        if r1 > r0:
            a = s["a"][r0:r1].double() * s["sa"][r0:r1].double()[:, kk]
            b = s["b"][e].double() * s["sb"][e].double()[nn][:, kk]
            z[r0:r1] = a @ b.t()
            if s["bias"]:
                z[r0:r1] += s["bias_v"][e].double()
    c = _act64(z, s["act"])[0]
    out = {"c": c if s["res"] is None else c + s["res"].double()}
    if s["pass"] == "saving":
        out["z"] = z
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": _exact_gate, "norm": _exact_norm, "matmul": _exact_matmul}[case["op"]](s)
