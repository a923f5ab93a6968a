"""Float64 references of the operators on expert rows, the gated activation and 8-bit checkpoints, and the
bounds of their fp32 errors. On torch tensors of any device; only what they name is shared with ops_ref."""
import math

import torch

from tests.ops_ref import U32

BLOCK = 32


def order(ids, E):
    """(slots, rows, offsets) by a walk over the slots."""
    flat = ids.reshape(-1).tolist()
    per = [[] for _ in range(E)]
    for slot, e in enumerate(flat):
        if 0 <= e < E:
            per[e].append(slot)
    slots = [s for p in per for s in p]
    rows = [-1] * len(flat)
    for r, s in enumerate(slots):
        rows[s] = r
    offsets = [0]
    for p in per:
        offsets.append(offsets[-1] + len(p))
    slots += [-1] * (len(flat) - len(slots))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(slots), i32(rows).view(ids.shape), i32(offsets)


def expert_rows(x, rows, n):
    out = torch.zeros(n, x.shape[-1], dtype=x.dtype, device=x.device)
    rows = rows.reshape(-1, rows.shape[-1])
    for j in range(rows.shape[1]):
        t = torch.nonzero(rows[:, j] >= 0)[:, 0]
        out[rows[t, j].long()] = x.reshape(-1, x.shape[-1])[t]
    return out


def taken(r, rows):
    """The rows of every slot [T, topk, D], zeros where there is none."""
    rows = rows.reshape(-1, rows.shape[-1])
    out = torch.zeros(*rows.shape, r.shape[-1], dtype=torch.float64, device=r.device)
    at = torch.nonzero(rows >= 0)
    out[at[:, 0], at[:, 1]] = r[rows[at[:, 0], at[:, 1]].long()].double()
    return out


def combine(r, w, rows):
    """(y, error): at most topk roundings of the running sum and one of each product."""
    got = taken(r, rows)
    terms = got if w is None else got * w.reshape(got.shape[:2])[:, :, None].double()
    return terms.sum(1), (rows.shape[-1] + 1) * U32 * terms.abs().sum(1)


def combine_backward(dy, r, w, rows, n):
    """(dr, dw, error of dw). A product's way through the sum of dw: D / 32 / warps / vector additions of
    a lane at most D / 32, five across the lanes, eight warps."""
    T, D = rows.reshape(-1, rows.shape[-1]).shape[0], dy.shape[-1]
    dy64, topk = dy.double().reshape(T, 1, D), rows.shape[-1]
    terms = taken(r, rows) * dy64
    w64 = w.double().reshape(T, topk)
    dr = torch.zeros(n, D, dtype=torch.float64, device=dy.device)
    flat = rows.reshape(T, topk)
    for j in range(topk):
        t = torch.nonzero(flat[:, j] >= 0)[:, 0]
        dr[flat[t, j].long()] = w64[t, j, None] * dy64[t, 0]
    return dr, terms.sum(2).view(rows.shape), (D / 32 + 5 + 8 + 2) * U32 * terms.abs().sum(2).view(rows.shape)


def products(x, w, offsets, add=None):
    """x[r] @ w[e] for w [E, K, N] in float64, and the sums of |x| |w|."""
    y = torch.zeros(x.shape[0], w.shape[2], dtype=torch.float64, device=x.device)
    size = torch.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        y[a:b] = x[a:b].double() @ w[e].double()
        size[a:b] = x[a:b].double().abs() @ w[e].double().abs()
    return (y if add is None else y + add.double()), size


def weights_grad(dy, x, offsets):
    """dW [E, N, K] in float64 and the sums of |dy| |x|."""
    E = len(offsets) - 1
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    size = torch.zeros_like(dw)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        dw[e] = dy[a:b].double().t() @ x[a:b].double()
        size[e] = dy[a:b].double().abs().t() @ x[a:b].double().abs()
    return dw, size


# The 127 numbers of e4m3 from 0 to 448: subnormal ones in steps of 2^-9, then eight to a binade.
E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119]


def encode(x):
    """(codes as numbers, 2^s) of a checkpoint of x [n, c] by search in the table: [n, c], [n, blocks]."""
    t = torch.tensor(E4M3, dtype=torch.float64)
    n, c = x.shape
    v = torch.nn.functional.pad(x.double().cpu(), (0, -c % BLOCK)).view(n, -1, BLOCK)
    finite = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))
    unit = torch.empty(n, v.shape[1], dtype=torch.float64)
    for i in range(n):
        for b, m in enumerate(finite[i].amax(1).tolist()):
            s = -127 if m == 0 else max(-127, math.frexp(m)[1] - 12)
            while m > 448 * 2.0 ** s:
                s += 1
            unit[i, b] = 2.0 ** s
    a = finite / unit[:, :, None]
    hi = torch.searchsorted(t, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = t[hi] - a, a - t[lo]
    at = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = torch.copysign(t[at], v)
    code = torch.where(torch.isfinite(v), code, torch.full_like(v, math.nan))
    return code.reshape(n, -1)[:, :c], unit


def decode(code, unit):
    return code * unit.repeat_interleave(BLOCK, 1)[:, :code.shape[1]]
