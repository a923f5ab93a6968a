"""Plain float64 (numpy) implementations of the operators around the routed experts, from
their formulas, for the tests of tile_signaled_grouped_gb300.ops. No library code here."""
import math

import numpy as np

U32 = 2.0 ** -24  # half a step of fp32


# ------------------------------------------------------------------------------- routing
def scores(l, score):
    l = np.asarray(l, dtype=np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    mx = l.max(axis=1, keepdims=True)
    e = np.where(np.isneginf(l), 0.0, np.exp(l - np.where(np.isneginf(mx), 0.0, mx)))
    return e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)


def route(l, topk, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1, renorm=False,
          scale=1.0):
    """(ids, weights) by sorting, one token at a time."""
    l = np.asarray(l, dtype=np.float64)
    n, E = l.shape
    s = scores(l, score)
    c = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    order = l if bias is None else c
    ids = np.empty((n, topk), dtype=np.int32)
    per = E // groups
    for t in range(n):
        ok = range(E)
        if groups > 1:
            best = [sum(sorted(c[t, g * per:(g + 1) * per], reverse=True)[:min(group_top, per)])
                    for g in range(groups)]
            keep = sorted(range(groups), key=lambda g: (-best[g], g))[:topk_groups]
            ok = [e for g in keep for e in range(g * per, (g + 1) * per)]
        ids[t] = sorted(ok, key=lambda e: (-order[t, e], e))[:topk]
    return ids, weights(l, ids, score, renorm, scale)


def weights(l, ids, score, renorm, scale):
    l = np.asarray(l, dtype=np.float64)
    s = np.take_along_axis(scores(l, score), ids.astype(np.int64), axis=1)
    if renorm:
        # the ratio of the scores from their logarithms, so that none underflows
        t = np.take_along_axis(l, ids.astype(np.int64), axis=1)
        if score == "sigmoid":
            t = np.minimum(t, 0.0) - np.log1p(np.exp(-np.abs(t)))
        m = t.max(axis=1, keepdims=True)
        e = np.where(np.isneginf(t), 0.0, np.exp(t - np.where(np.isneginf(m), 0.0, m)))
        S = e.sum(axis=1, keepdims=True)
        s = np.where(S > 0, e / np.where(S > 0, S, 1.0), 0.0)
    return scale * s


def route_backward(dw, l, ids, score, renorm, scale):
    l = np.asarray(l, dtype=np.float64)
    dw = np.asarray(dw, dtype=np.float64)
    at = ids.astype(np.int64)
    r = weights(l, ids, score, renorm, 1.0)
    g = scale * dw
    s = scores(l, score)
    d = np.zeros_like(l)
    if renorm:
        v = r * (g - (g * r).sum(axis=1, keepdims=True))
        if score == "sigmoid":
            v = v * (1.0 - np.take_along_axis(s, at, axis=1))
        np.put_along_axis(d, at, v, axis=1)
    elif score == "sigmoid":
        np.put_along_axis(d, at, g * r * (1.0 - np.take_along_axis(s, at, axis=1)), axis=1)
    else:
        np.put_along_axis(d, at, g, axis=1)
        d = s * (d - (g * r).sum(axis=1, keepdims=True))
    return d


def weight_tolerance(l, k):
    """Relative error of a weight in fp32, in half steps: 4 for expf (2 ulp), 1 for each
    addition of a sum (at most 32 of a lane's and 5 across lanes, or 5 of the chosen), the
    rounded argument of the exponential (the range of the scores, in the numerator and in
    the sum) and a division, a product and the scale."""
    f = np.where(np.isfinite(l), l, np.nan)
    span = float(np.nanmax(f) - np.nanmin(f)) if np.isfinite(l).any() else 0.0
    return U32 * (2 * span + 4 + 4 + 37 + 5 + 8)


# ---------------------------------------------------------------------------- layer norm
def layer_norm(x, w, b, eps, r=None):
    """(y, z, mean, rstd) in float64."""
    z = x if r is None else x + r
    mean = z.mean(axis=1)
    d = z - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    y = y if w is None else y * w
    return (y if b is None else y + b), z, mean, rstd


def layer_norm_backward(dy, z, w, mean, rstd, dz=None):
    """(dx, dw, db) in float64."""
    xhat = (z - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) -
                          xhat * (g * xhat).mean(axis=1, keepdims=True))
    return (dx if dz is None else dx + dz), (dy * xhat).sum(axis=0), dy.sum(axis=0)


def chain(D):
    """Additions that one value passes through in a sum of D: at most 32 in a thread (or D /
    1024 and a vector in the long-row kernels) and 10 across the warps of a CTA."""
    return 32 + 10 + D / 1024 + 8


def layer_norm_tolerance(x, w, b, eps, r=None):
    """Bounds of the fp32 errors of (y, z, mean, rstd), before y and z are rounded."""
    y, z, mean, rstd = layer_norm(x, w, b, eps, r)
    c, D = chain(x.shape[1]), x.shape[1]
    ez = U32 * np.abs(z) if r is not None else np.zeros_like(z)
    em = (c + 2) * U32 * np.abs(z).mean(axis=1) + ez.mean(axis=1)
    d = np.abs(z - mean[:, None])
    ed = ez + em[:, None] + U32 * d
    # var: each square moves by 2 d ed + ed^2; the sum by c roundings; sqrt halves it.
    ev = (2 * d * ed + ed * ed).mean(axis=1) + (c + 3) * U32 * (d * d).mean(axis=1)
    rel = 0.5 * ev * rstd * rstd * (1 + ev * rstd * rstd) + 4 * U32
    aw = 1.0 if w is None else np.abs(w)
    ab = 0.0 if b is None else np.abs(b)
    ey = aw * (ed * rstd[:, None] * (1 + rel[:, None]) + d * rstd[:, None] * (rel[:, None] + 3 * U32))
    return ey + U32 * (np.abs(y) + ab), ez, em + U32 * np.abs(mean), rel * rstd


def layer_norm_backward_tolerance(dy, z, w, mean, rstd, dz=None):
    """Bounds of the fp32 errors of (dx, dw, db), before they are rounded."""
    c, n = chain(z.shape[1]), z.shape[0]
    xhat = np.abs((z - mean[:, None]) * rstd[:, None])
    g = np.abs(dy) if w is None else np.abs(dy * w)
    m1, m2 = g.mean(axis=1, keepdims=True), (g * xhat).mean(axis=1, keepdims=True)
    ex = rstd[:, None] * U32 * (4 * g + (c + 6) * m1 + (c + 12) * xhat * m2)
    if dz is not None:
        ex = ex + 2 * U32 * np.abs(dz)
    # Rows: n / 304 of a thread (at least 152 CTAs where there are that many rows), eight
    # row groups of a CTA, 304 / 8 of the CTAs, and eight warps.
    rows = n / 152 + 8 + 38 + 8 + 4
    return ex, rows * U32 * (np.abs(dy) * xhat).sum(axis=0), rows * U32 * np.abs(dy).sum(axis=0)


# -------------------------------------------------------------------------------- linear
# On float64 torch tensors (any device), since the sizes are larger here.
def _t():
    import torch

    return torch


C0, C1 = math.sqrt(2.0 / math.pi), 0.044715


def act(z, kind):
    t = _t()
    if kind == "relu":
        return t.where(z > 0, z, t.zeros_like(z))
    if kind == "gelu":
        return 0.5 * z * t.special.erfc(-z * math.sqrt(0.5))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + t.tanh(C0 * (z + C1 * z ** 3)))
    if kind == "silu":
        return z / (1 + t.exp(-z))
    return z


def act_grad(z, kind):
    t = _t()
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * t.special.erfc(-z * math.sqrt(0.5)) + z * t.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        th = t.tanh(C0 * (z + C1 * z ** 3))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * C0 * (1 + 3 * C1 * z * z)
    if kind == "silu":
        s = 1 / (1 + t.exp(-z))
        return s * (1 + z * (1 - s))
    return t.ones_like(z)


def act_error(z, kind):
    """Absolute fp32 errors of act(z) and act'(z). The fast exponential is within 2 + 1.2 |v|
    steps of its argument v, the fast division within 2, erff within 2; the argument itself
    carries four roundings."""
    v = z.abs()
    if kind == "gelu_tanh":
        v = 2 * C0 * (v + C1 * v ** 3)
    if kind in ("none", "relu"):
        return 0 * v, 0 * v
    v = v.clamp(max=45.0)  # beyond, the sigmoid is 0 or 1
    steps = 32 + 16 * v
    return act(z, kind).abs() * steps * U32 + 8 * U32 * z.abs(), steps * U32 * (1 + z.abs().clamp(max=30.0))


def product_error(a, b, k):
    """Of a @ b with k fp32 additions in any order: two half steps each, for sums that the
    tensor cores cut off rather than round."""
    return 2 * (k + 24) * U32 * (a.abs() @ b.abs())
