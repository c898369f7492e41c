"""Router, tokens to rows and back, and FP8 with a scale per block of 128.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Everything is computed from its definition in float64, except the quantizer,
whose definition is three fp32 steps (scale, its reciprocal, product) and is
computed in exactly those.  ``dst`` is the row of each choice, -1 for a
dropped one; ``w`` None stands for ones.
"""
import numpy as np

from . import formats as F
from . import swiglu as S

BLOCK = 128
F32 = np.float32


# ------------------------------------------------------------------ router

def gate_topk(x, k, normalize, scale):
    """(ids int32 [T, k], weights float64 [T, k]): the k largest logits, ties
    to the lowest index, -inf and NaN never chosen (-1, weight 0)."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        ok = [j for j in range(E) if x[t, j] > -np.inf]           # False for NaN
        best = sorted(ok, key=lambda j: (-x[t, j], j))[:k]
        ids[t, :len(best)] = best
        if not best:
            continue
        m = x[t, best[0]]
        if np.isnan(x[t]).any() or np.isinf(m):
            w[t] = np.nan
            continue
        e = np.exp(x[t] - m)
        total = e[best].sum() if normalize else e.sum()
        w[t, :len(best)] = scale * e[best] / total
    return ids, w


def gate_topk_grad(x, ids, dw, normalize, scale):
    """d_logits float64 [T, E] from the softmax's Jacobian, the choice fixed."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    dx = np.zeros((T, E))
    for t in range(T):
        at = [(int(i), r) for r, i in enumerate(ids[t]) if i >= 0]
        if not np.isfinite(x[t].max()):
            continue
        over = sorted({i for i, _ in at}) if normalize else list(range(E))
        if not over:
            continue
        e = np.exp(x[t, over] - x[t].max())
        p = e / e.sum()
        place = {j: n for n, j in enumerate(over)}
        g = np.zeros(len(over))
        for i, r in at:
            g[place[i]] += scale * float(dw[t, r])
        dx[t, over] = (np.diag(p) - np.outer(p, p)) @ g if len(over) <= 64 else p * (g - p @ g)
    return dx


# ------------------------------------------------- tokens, rows, gradients

def spread(x, dst, w, total_rows):
    """rows float64 [total_rows, H], NaN where no choice writes."""
    rows = np.full((total_rows, x.shape[1]), np.nan)
    for t, j in np.ndindex(*dst.shape):
        if dst[t, j] >= 0:
            rows[dst[t, j]] = x[t].astype(np.float64) * (1.0 if w is None else float(w[t, j]))
    return rows


def collect(rows, dst, w):
    """(sums float64 [T, H], sums of magnitudes)."""
    T, k = dst.shape
    y = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(y)
    for t, j in np.ndindex(T, k):
        if dst[t, j] >= 0:
            v = rows[dst[t, j]].astype(np.float64) * (1.0 if w is None else float(w[t, j]))
            y[t] += v
            mag[t] += np.abs(v)
    return y, mag


def dots(x, rows, dst):
    """(d_w float64 [T, k], sums of magnitudes)."""
    d = np.zeros(dst.shape)
    mag = np.zeros(dst.shape)
    for t, j in np.ndindex(*dst.shape):
        if dst[t, j] >= 0:
            v = x[t].astype(np.float64) * rows[dst[t, j]].astype(np.float64)
            d[t, j], mag[t, j] = v.sum(), np.abs(v).sum()
    return d, mag


# ----------------------------------------------------- FP8 with 128-blocks

def _codes(x, amax):
    """E4M3 codes and scale of one block of fp32 values."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        s = np.maximum(F32(amax) / F32(448.0), F32(2.0 ** -126))
        v = x.astype(F32) * (F32(1.0) / s)
    q = F.encode_e4m3(np.where(np.isnan(v), 0.0, v))
    return np.where(np.isnan(v), np.uint8(0x7F), q), s


def _amax(x):
    m = np.abs(x[~np.isnan(x)])
    return m.max() if m.size else F32(0.0)


def quantize_rows(x):
    """x fp32 [R, K] -> (codes uint8 [R, K], scales fp32 [R, ceil(K / 128)])."""
    x = np.asarray(x, F32)
    R, K = x.shape
    q = np.zeros((R, K), np.uint8)
    s = np.zeros((R, -(-K // BLOCK)), F32)
    for r, b in np.ndindex(*s.shape):
        part = x[r, b * BLOCK:(b + 1) * BLOCK]
        q[r, b * BLOCK:(b + 1) * BLOCK], s[r, b] = _codes(part, _amax(part))
    return q, s


def quantize_weight(w):
    """w fp32 [E, N, K] -> (codes, scales fp32 [E, ceil(N / 128), ceil(K / 128)])."""
    w = np.asarray(w, F32)
    E, N, K = w.shape
    q = np.zeros((E, N, K), np.uint8)
    s = np.zeros((E, -(-N // BLOCK), -(-K // BLOCK)), F32)
    for e, n, k in np.ndindex(*s.shape):
        at = (e, slice(n * BLOCK, (n + 1) * BLOCK), slice(k * BLOCK, (k + 1) * BLOCK))
        q[at], s[e, n, k] = _codes(w[at], _amax(w[at]))
    return q, s


def swiglu_quantize(y):
    """y fp32 [R, 2 I], gate in the even columns; h as the library defines it."""
    y = np.asarray(y, F32)
    return quantize_rows(S.swiglu(y))


def matmul(a, b, sa, sb, offsets, expert_ids):
    """float64 [T, N], NaN where no group writes."""
    T, K = a.shape
    E, N, _ = b.shape
    kk, nn = np.arange(K) // BLOCK, np.arange(N) // BLOCK
    c = np.full((T, N), np.nan)
    for g, e in enumerate(expert_ids):
        r0, r1 = int(offsets[g]), int(offsets[g + 1])
        if r1 > r0:
            av = F.decode_e4m3(a[r0:r1]) * np.asarray(sa[r0:r1], np.float64)[:, kk]
            bv = F.decode_e4m3(b[e]) * np.asarray(sb[e], np.float64)[nn][:, kk]
            c[r0:r1] = av @ bv.T
    return c
