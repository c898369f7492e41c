"""The scored and grouped router, the residual's addition with the
root-mean-square norm, and the epilogue of the FP8 block product.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Everything is computed from its definition in float64; what the definition
rounds on the way (the residual stream, the saved pre-activation) is given to
these functions rounded.
"""
import math

import numpy as np

BLOCK = 128
NONE = -np.inf


# ------------------------------------------------------------------ router

def scores(x, kind):
    """s of each logit, float64; NaN everywhere where a softmax is none."""
    x = np.asarray(x, np.float64)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    out = np.full(x.shape, np.nan)
    for t in range(x.shape[0]):
        m = x[t].max()                       # NaN where there is one
        if np.isfinite(m):
            e = np.exp(x[t] - m)
            out[t] = e / e.sum()
        elif m == NONE:
            out[t] = 0.0
    return out


def gate_group_topk(x, k, bias=None, score="sigmoid", groups=1, topk_groups=None,
                    group_score="top2", normalize=True, scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k])."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    size, some = E // groups, topk_groups or groups
    s = scores(x, score)
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        nan = bool(np.isnan(x[t]).any())
        plain = score == "softmax" and np.isnan(s[t]).any()      # by the logits alone
        c = np.full(E, NONE)                 # what orders the experts
        v = np.full(E, NONE)                 # what the groups sum
        for j in range(E):
            if not x[t, j] > NONE:
                continue
            if bias is None or plain:
                c[j], v[j] = x[t, j], s[t, j]
            else:
                c[j] = v[j] = s[t, j] + float(bias[j])
                if not c[j] > NONE:
                    c[j] = v[j] = NONE
        value = np.full(groups, NONE)
        for g in range(groups):
            part = slice(g * size, (g + 1) * size)
            if plain or group_score == "max":
                value[g] = c[part].max()
            else:
                best = sorted(v[part], reverse=True)[:2]
                value[g] = best[0] + best[1] if len(best) > 1 and best[1] > NONE else best[0]
        kept = set(sorted(range(groups), key=lambda g: (-value[g], g))[:some])
        order = sorted((j for j in range(E) if c[j] > NONE and j // size in kept),
                       key=lambda j: (-c[j], j))[:k]
        ids[t, :len(order)] = order
        if not order:
            continue
        if nan or plain:
            w[t] = np.nan
            continue
        top = s[t, order]
        if normalize and score == "softmax":
            e = np.exp(x[t, order] - x[t, order].max())          # the denominator cancels
            top = e / e.sum()
        elif normalize:
            top = top / top.sum() if top.sum() > 0 else top * 0.0
        w[t, :len(order)] = scale * top
    return ids, w


def gate_group_topk_grad(x, ids, dw, score, normalize, scale):
    """d_logits float64 [T, E] through the weights' Jacobian, the choice fixed."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    dx = np.zeros((T, E))
    s = scores(x, score)
    for t in range(T):
        at = [(int(i), r) for r, i in enumerate(ids[t]) if i >= 0]
        if not at:
            continue
        j = [i for i, _ in at]
        g = np.array([scale * float(dw[t, r]) for _, r in at])
        if normalize:
            total = s[t, j].sum()
            if not total > 0:
                continue
            q = s[t, j] / total
            ds = (g - (q * g).sum()) / total
        else:
            ds = g
        full = np.zeros(E)
        full[j] = ds
        if score == "sigmoid":
            dx[t] = full * s[t] * (1.0 / (1.0 + np.exp(x[t])))
        else:
            dx[t] = s[t] * (full - (s[t] * full).sum())
    return dx


# -------------------------------------------------------------------- norm

def rms_norm(h, w, eps):
    """(y, 1 / rms) float64 of rows h."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def rms_norm_grad(h, w, eps, dy, dh=None):
    """(d_x, d_weight, magnitudes of d_weight's terms) float64."""
    h, w, dy = (np.asarray(v, np.float64) for v in (h, w, dy))
    _, rstd = rms_norm(h, w, eps)
    unit = h * rstd[:, None]
    g = dy * w
    dx = (g - unit * (g * unit).mean(1, keepdims=True)) * rstd[:, None]
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * unit).sum(0), np.abs(dy * unit).sum(0)


# ---------------------------------------------------------------- epilogue

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activate(z, name):
    """(act(z), its slope) float64."""
    z = np.asarray(z, np.float64)
    one = np.ones_like(z)
    if name is None:
        return z, one
    if name == "relu":
        return np.maximum(z, 0.0), np.where(np.isnan(z), z, (z > 0) * one)
    if name == "silu":
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    if name == "gelu":
        c = 0.5 * (1.0 + _erf(z / np.sqrt(2.0)))
        return z * c, c + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    assert name == "gelu_tanh"
    a = np.sqrt(2.0 / np.pi)
    t = np.tanh(a * (z + 0.044715 * z ** 3))
    return (0.5 * z * (1.0 + t),
            0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z))


def row_experts(offsets, expert_ids, rows):
    """The expert of each row, -1 outside every group."""
    e = np.full(rows, -1, np.int64)
    for g, i in enumerate(expert_ids):
        e[int(offsets[g]):int(offsets[g + 1])] = i
    return e


def epilogue(z, name, residual=None):
    c = activate(z, name)[0]
    return c if residual is None else c + np.asarray(residual, np.float64)


def epilogue_grad(dc, z, name, experts, num_experts):
    """(dz, d_bias [num_experts, N], magnitudes of its terms) float64."""
    dz = np.asarray(dc, np.float64) * (1.0 if z is None else activate(z, name)[1])
    db = np.zeros((num_experts, dz.shape[1]))
    mag = np.zeros_like(db)
    for r, e in enumerate(experts):
        if e >= 0:
            db[e] += dz[r]
            mag[e] += np.abs(dz[r])
    return dz, db, mag
