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
