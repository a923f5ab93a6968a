"""The operators around the routed experts of a transformer block, as cases to measure: routing to
experts from their scores, layer norm (with the sum of a residual stream) and the matrix product with
bias, activation and residual, each forward and backward.

A case is a dict of plain values; "op" says which operator and direction:
  route       ids and weights of the topk experts of every token from its scores
  route_grad  the gradient of the scores from the gradient of the weights
  norm        z = x + r, y = (z - mean) / sqrt(var + eps) * weight + bias
  norm_grad   the gradients of z, weight and bias
  linear      y = act(x W^T + b) + r
  linear_grad the gradients of x, W and b

With own = False, run() computes them in elementary torch operations; with own = True it calls
tile_signaled_grouped_gb300.ops. exact() computes them in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def _route(name, op, n, E, topk, score, bias=False, groups=1, topk_groups=1, group_top=1,
           renorm=False, scale=1.0, mask=False, pad=0, dtype="fp32"):
    return dict(name=name, op=op, n=n, E=E, topk=topk, score=score, bias=bias, groups=groups,
                topk_groups=topk_groups, group_top=group_top, renorm=renorm, scale=scale, mask=mask,
                pad=pad, dtype=dtype)


def _norm(name, op, n, D, dtype, wtype, residual=False, beta=True, pad=0, stats=False):
    return dict(name=name, op=op, n=n, D=D, dtype=dtype, wtype=wtype, residual=residual, beta=beta,
                pad=pad, stats=stats)


def _linear(name, op, M, N, K, dtype, act="none", bias=True, btype="fp32", residual=False, pad=0,
            preact=False):
    return dict(name=name, op=op, M=M, N=N, K=K, dtype=dtype, act=act, bias=bias, btype=btype,
                residual=residual, pad=pad, preact=preact)


def listed():
    return [
        # One token of a decoding step through a router of 256 experts in 8 groups: latency.
        _route("route one token", "route", 1, 256, 8, "sigmoid", bias=True, groups=8, topk_groups=4,
               group_top=2, renorm=True, scale=2.5),
        # A ragged batch of a softmax router whose score matrix is the 16-bit output of a product
        # and stands in wider rows; some experts are masked, and all of some rows.
        _route("route ragged masked", "route", 1001, 120, 6, "softmax", renorm=True, mask=True,
               pad=8, dtype="bf16"),
        # A long prompt, or a training batch, through the 256-expert router.
        _route("route prompt", "route", 16384, 256, 8, "sigmoid", bias=True, groups=8,
               topk_groups=4, group_top=2, renorm=True, scale=2.5),
        # Its training step: softmax over 128 experts, weights not renormalised.
        _route("route gradient", "route_grad", 16384, 128, 8, "softmax"),
        # One token's norm at the widest model size here: latency.
        _norm("norm one token", "norm", 1, 7168, "bf16", "bf16", residual=True),
        # Odd rows of an odd length inside wider rows.
        _norm("norm ragged", "norm", 777, 1531, "fp16", "fp32", beta=False, pad=5, stats=True),
        # The norm of a prompt, with the residual stream's sum.
        _norm("norm prompt", "norm", 16384, 4096, "bf16", "bf16", residual=True, stats=True),
        # The norm's backward pass over a training batch.
        _norm("norm gradient", "norm_grad", 8192, 7168, "bf16", "fp32", residual=True),
        # One token through the first matrix of a dense expert: reads the weights once.
        _linear("linear one token", "linear", 1, 2048, 7168, "bf16", act="silu"),
        # A ragged batch back to an odd width, with the residual.
        _linear("linear ragged", "linear", 333, 517, 1000, "fp16", act="gelu", btype="fp16",
                residual=True, pad=8),
        # A training batch or prompt through the first matrix of a dense expert.
        _linear("linear prompt", "linear", 8192, 8192, 2048, "bf16", act="gelu_tanh", preact=True),
        # The backward pass of such a matrix.
        _linear("linear gradient", "linear_grad", 4096, 1536, 4096, "bf16", act="silu"),
    ]


def _count(rng, most):
    """1 to `most` tokens, even in the logarithm: a power of two, or an odd number."""
    v = min(math.exp(rng.uniform(0.0, math.log(16384))), most)
    return 1 << int(math.log2(v)) if rng.random() < 0.4 else max(1, int(v) - 1 + int(v) % 2)


def draw(rng):
    """A case of the ranges that the listed ones stand for: any operator, 1 to 16384 tokens."""
    op = rng.choice(["route", "route_grad", "norm", "norm_grad", "linear", "linear_grad"])
    if op.startswith("route"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.choice([2, 3, 5, 8, 16, 32]) if groups > 1 else rng.choice(
            [8, 16, 128, 256, rng.randint(9, 255)])
        tg = rng.randint(max(1, groups // 2), groups)
        topk = rng.randint(1, min(8, tg * (E // groups)))
        # One expert's renormalised weight is the constant `scale`, and its gradient zero.
        renorm = rng.random() < 0.5 and not (op == "route_grad" and topk == 1)
        return dict(op=op, n=_count(rng, 16384), E=E, topk=topk,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=tg, group_top=rng.choice([1, 2]), renorm=renorm, scale=rng.choice([1.0, 2.5]), mask=groups == 1 and rng.random() < 0.3,
                    pad=rng.choice([0, 0, 3, 8]), dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]))
    if op.startswith("norm"):
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        D = rng.choice([128, 1536, 2048, 4096, 5120, 7168, 2 * rng.randint(20, 4095) + 1])
        return dict(op=op, n=_count(rng, (1 << 25) // D), D=D, dtype=dtype,
                    wtype=rng.choice([dtype, "fp32"]), residual=rng.random() < 0.5,
                    beta=rng.random() < 0.7, pad=rng.choice([0, 0, 5, 8]), stats=rng.random() < 0.5)
    N = rng.choice([128, 256, 1536, 2048, 4096, 8192, 2 * rng.randint(8, 4095) + 1])
    K = rng.choice([128, 256, 1536, 2048, 4096, 7168, 8 * (2 * rng.randint(1, 511) + 1)])
    most = 4096 * 4096 * 1536 if op == "linear_grad" else 8192 * 8192 * 2048
    dtype = rng.choice(["bf16", "fp16"])
    return dict(op=op, M=_count(rng, max(1, min(8192, most // (N * K)))), N=N, K=K,
                dtype=dtype, act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                bias=rng.random() < 0.8, btype=rng.choice([dtype, "fp32"]),
                residual=op == "linear" and rng.random() < 0.5, pad=rng.choice([0, 0, 8]),
                preact=op == "linear" and rng.random() < 0.3)


# ------------------------------------------------------------------------------------- inputs
class _Maker:
    """Seeded tensors on the GPU."""

    def __init__(self, seed):
        self.dev = "cuda" if torch.cuda.is_available() else "cpu"
        self.g = torch.Generator(device=self.dev)
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, mean=0.0):
        return torch.empty(shape, device=self.dev).normal_(mean, std, generator=self.g)

    def uniform(self, *shape):
        return torch.rand(shape, device=self.dev, generator=self.g)

    def rows(self, values, dtype, pad):
        """`values` in `dtype`, as the first columns of rows that are `pad` elements wider."""
        n, c = values.shape
        t = torch.zeros(n, c + pad, dtype=dtype, device=self.dev)
        t[:, :c] = values.to(dtype)
        return t[:, :c]


def _inputs(case, seed):
    mk = _Maker(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    s = dict(case)
    if op.startswith("route"):
        n, E, k = case["n"], case["E"], case["topk"]
        logits = mk.normal(n, E, std=1.5)
        if case["mask"]:
            logits.masked_fill_(mk.uniform(n, E) < 0.2, -math.inf)
            logits[mk.uniform(n) < 0.02] = -math.inf
        s["logits"] = mk.rows(logits, dt, case["pad"])
        s["b"] = mk.normal(E, std=0.1) if case["bias"] else None
        if op == "route_grad":
            s["ids"] = _route_ids(s)  # saved by the forward pass
            s["dw"] = mk.normal(n, k)
        return s
    if op.startswith("norm"):
        n, D, wt = case["n"], case["D"], TYPES[case["wtype"]]
        # Channels of different size and offset, as hidden states have them.
        x = mk.normal(n, D) * torch.exp(mk.normal(D, std=0.5)) + mk.normal(D, std=0.5) + 0.3
        s["w"] = (1.0 + 0.2 * mk.normal(D)).to(wt)
        if op == "norm":
            s["x"] = mk.rows(x, dt, case["pad"])
            s["b"] = (0.2 * mk.normal(D)).to(wt) if case["beta"] else None
            s["r"] = mk.rows(mk.normal(n, D), dt, case["pad"]) if case["residual"] else None
        else:
            s["z"] = mk.rows(x, dt, case["pad"])
            s["dy"] = mk.rows(mk.normal(n, D), dt, case["pad"])
            s["dz"] = mk.rows(mk.normal(n, D), dt, case["pad"]) if case["residual"] else None
            z = s["z"].float()  # saved by the forward pass
            s["mean"] = z.mean(1)
            s["rstd"] = 1.0 / torch.sqrt((z - s["mean"][:, None]).square().mean(1) + EPS)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s["x"] = mk.rows(mk.normal(M, K), dt, case["pad"])
    s["w"] = mk.rows(mk.normal(N, K, std=1.0 / math.sqrt(K)), dt, case["pad"])
    if op == "linear":
        s["b"] = mk.normal(N, std=0.2).to(TYPES[case["btype"]]) if case["bias"] else None
        s["r"] = mk.rows(mk.normal(M, N), dt, case["pad"]) if case["residual"] else None
    else:
        s["dy"] = mk.rows(mk.normal(M, N), dt, 8 - N % 8 if N % 8 else case["pad"])
        # The product before the activation, saved by the forward pass.
        s["z"] = mk.rows(mk.normal(M, N), dt, case["pad"]) if case["act"] != "none" else None
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---------------------------------------------------------------------------------- plain form
def _route_ids(s):
    """The topk ids: in 64 bits, since two experts' scores may lie within a rounding of 32."""
    l, E, G, k = s["logits"].double(), s["E"], s["groups"], s["topk"]
    if s["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True).clamp(min=-1e300))
        c = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        c = 1.0 / (1.0 + torch.exp(-l))
    if s["b"] is not None:
        c = c + s["b"].double()
    if G > 1:
        per = c.view(-1, G, E // G)
        best = per.sort(dim=2, descending=True).values[:, :, :min(s["group_top"], E // G)].sum(2)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        out = torch.ones_like(best, dtype=torch.bool).scatter_(1, keep, False)
        c = per.masked_fill(out[:, :, None], -math.inf).view(-1, E)
    return c.sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)


def _scores(s):
    """The experts' probabilities in 32 bits; 0 for a masked expert."""
    l = s["logits"].float()
    if s["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True).clamp(min=-1e38))
    return e / e.sum(1, keepdim=True).clamp(min=1e-38)


def _route_plain(s):
    ids = _route_ids(s)
    w = _scores(s).gather(1, ids.long())
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-38)
    return {"ids": ids, "w": w * s["scale"]}


def _route_grad_plain(s):
    p, at = _scores(s), s["ids"].long()
    dw = s["dw"] * s["scale"]
    if s["renorm"]:
        c = p.gather(1, at)
        S = c.sum(1, keepdim=True).clamp(min=1e-38)
        dw = (dw - (dw * c).sum(1, keepdim=True) / S) / S
    dp = torch.zeros_like(p).scatter_(1, at, dw)
    if s["score"] == "sigmoid":
        d = dp * p * (1.0 - p)
    elif s["renorm"]:
        d = dp * p  # the sum of dp p over the chosen experts is zero
    else:
        d = p * (dp - (dp * p).sum(1, keepdim=True))
    return {"d_logits": d.to(s["logits"].dtype)}


def _norm_plain(s):
    x = s["x"]
    z = x.float() if s["r"] is None else x.float() + s["r"].float()
    mean = z.mean(1)
    c = z - mean[:, None]
    rstd = 1.0 / torch.sqrt(c.square().mean(1) + EPS)
    y = c * rstd[:, None] * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    out = {"y": y.to(x.dtype)}
    if s["r"] is not None:
        out["z"] = z.to(x.dtype)
    if s["stats"]:
        out.update(mean=mean, rstd=rstd)
    return out


def _norm_grad_plain(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["z"].float() - s["mean"][:, None]) * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dz"] is not None:
        dx = dx + s["dz"].float()
    out = {"dx": dx.to(s["z"].dtype), "dw": (dy * xhat).sum(0).to(s["w"].dtype)}
    if s["beta"]:
        out["db"] = dy.sum(0).to(s["w"].dtype)
    return out


_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "relu":
        return torch.maximum(z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_C0 * (z + _C1 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(
            2.0 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_C0 * (z + _C1 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C0 * (1.0 + 3.0 * _C1 * z * z)
    q = 1.0 / (1.0 + torch.exp(-z))
    return q * (1.0 + z * (1.0 - q))


def _linear_plain(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"y": y.to(s["x"].dtype)}
    if s["preact"]:
        out["z"] = z.to(s["x"].dtype)
    return out


def _linear_grad_plain(s):
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_grad(s["z"].float(), s["act"])
    out = {"dx": (dz @ s["w"].float()).to(s["x"].dtype),
           "dw": (dz.t() @ s["x"].float()).to(s["w"].dtype)}
    if s["bias"]:
        out["db"] = dz.sum(0).to(TYPES[s["btype"]])
    return out


# ------------------------------------------------------------------------------- the framework
def _run_own(s):
    from tile_signaled_grouped_gb300 import ops

    op = s["op"]
    if op == "route":
        ids, w = ops.route_experts(s["logits"], s["topk"], score=s["score"], bias=s["b"],
                                   groups=s["groups"], topk_groups=s["topk_groups"],
                                   group_top=s["group_top"], renorm=s["renorm"], scale=s["scale"])
        return {"ids": ids, "w": w}
    if op == "route_grad":
        return {"d_logits": ops.route_experts_backward(s["dw"], s["logits"], s["ids"],
                                                       score=s["score"], renorm=s["renorm"],
                                                       scale=s["scale"])}
    if op == "norm":
        y, z, mean, rstd = ops.layer_norm(s["x"], s["w"], s["b"], eps=EPS, residual=s["r"],
                                          stats=s["stats"])
        out = {"y": y}
        if s["r"] is not None:
            out["z"] = z
        if s["stats"]:
            out.update(mean=mean, rstd=rstd)
        return out
    if op == "norm_grad":
        dx, dw, db = ops.layer_norm_backward(s["dy"], s["z"], s["w"], s["mean"], s["rstd"],
                                             dz=s["dz"], bias=s["beta"])
        return {"dx": dx, "dw": dw, "db": db} if s["beta"] else {"dx": dx, "dw": dw}
    if op == "linear":
        y, z = ops.linear(s["x"], s["w"], s["b"], act=s["act"], residual=s["r"], preact=s["preact"])
        return {"y": y, "z": z} if s["preact"] else {"y": y}
    dx, dw, db = ops.linear_backward(s["dy"], s["x"], s["w"], z=s["z"], act=s["act"],
                                     bias=TYPES[s["btype"]] if s["bias"] else None)
    return {"dx": dx, "dw": dw, "db": db} if s["bias"] else {"dx": dx, "dw": dw}


def run(state):
    if own:
        return _run_own(state)
    return {"route": _route_plain, "route_grad": _route_grad_plain, "norm": _norm_plain,
            "norm_grad": _norm_grad_plain, "linear": _linear_plain,
            "linear_grad": _linear_grad_plain}[state["op"]](state)


def work(case):
    """Each input read once and each output written once; the operations of the products, and of
    the elementwise parts a handful for each element."""
    op, e = case["op"], BYTES[case["dtype"]]
    if op.startswith("route"):
        n, E, k = case["n"], case["E"], case["topk"]
        if op == "route":
            return {"bytes": n * E * e + n * k * 8 + (4 * E if case["bias"] else 0), "flops": 10 * n * E}
        read = n * E * e if case["score"] == "softmax" and not case["renorm"] else n * k * e
        return {"bytes": read + n * E * e + n * k * 8, "flops": 10 * n * E}
    if op.startswith("norm"):
        n, D, we = case["n"], case["D"], BYTES[case["wtype"]]
        if op == "norm":
            return {"bytes": n * D * e * (4 if case["residual"] else 2) +
                    D * we * (2 if case["beta"] else 1) + (8 * n if case["stats"] else 0),
                    "flops": 8 * n * D}
        return {"bytes": n * D * e * (4 if case["residual"] else 3) +
                D * we * (3 if case["beta"] else 2) + 8 * n, "flops": 14 * n * D}
    M, N, K = case["M"], case["N"], case["K"]
    bias = N * BYTES[case["btype"]] if case["bias"] else 0
    if op == "linear":
        rows = 1 + (1 if case["residual"] else 0) + (1 if case["preact"] else 0)
        return {"bytes": e * (M * K + N * K + rows * M * N) + bias, "flops": 2 * M * N * K}
    rows = 2 if case["act"] != "none" else 1
    return {"bytes": e * (2 * M * K + 2 * N * K + rows * M * N) + bias, "flops": 4 * M * N * K}


# ------------------------------------------------------------------------------ 64-bit results
def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    F = torch.nn.functional
    if op.startswith("route"):
        l = s["logits"].double().requires_grad_(op == "route_grad")
        logp = F.logsigmoid(l) if case["score"] == "sigmoid" else F.log_softmax(l, 1)
        if op == "route":
            at = _exact_ids(case, s)
        else:
            at = s["ids"].long()
        t = logp.gather(1, at)
        # A renormalised weight is the softmax of the chosen experts' log scores.
        w = case["scale"] * (torch.softmax(t, 1) if case["renorm"] else torch.exp(t))
        if op == "route":
            return {"ids": at.to(torch.int32), "w": torch.nan_to_num(w, nan=0.0)}
        (d,) = torch.autograd.grad(w, l, s["dw"].double())
        return {"d_logits": torch.nan_to_num(d, nan=0.0)}
    if op == "norm":
        z = s["x"].double() + (0 if s["r"] is None else s["r"].double())
        w, b = s["w"].double(), None if s["b"] is None else s["b"].double()
        out = {"y": F.layer_norm(z, (case["D"],), w, b, EPS)}
        if s["r"] is not None:
            out["z"] = z
        if case["stats"]:
            var, mean = torch.var_mean(z, 1, correction=0)
            out.update(mean=mean, rstd=(var + EPS).rsqrt())
        return out
    if op == "norm_grad":
        z = s["z"].double().requires_grad_()
        w = s["w"].double().requires_grad_()
        b = torch.zeros_like(w).requires_grad_()
        # The statistics are the saved ones, and the gradient flows through them.
        dz, dw, db = torch.autograd.grad(F.layer_norm(z, (case["D"],), w, b, EPS), (z, w, b),
                                         s["dy"].double())
        if s["dz"] is not None:
            dz = dz + s["dz"].double()
        return {"dx": dz, "dw": dw, "db": db} if case["beta"] else {"dx": dz, "dw": dw}
    act = {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
           "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[case["act"]]
    x, w = s["x"].double(), s["w"].double()
    if op == "linear":
        z = F.linear(x, w, None if s["b"] is None else s["b"].double())
        y = act(z) if s["r"] is None else act(z) + s["r"].double()
        return {"y": y, "z": z} if case["preact"] else {"y": y}
    dz = s["dy"].double()
    if s["z"] is not None:
        z = s["z"].double().requires_grad_()
        (dz,) = torch.autograd.grad(act(z), z, dz)
    out = {"dx": torch.einsum("mn,nk->mk", dz, w), "dw": torch.einsum("mn,mk->nk", dz, x)}
    if case["bias"]:
        out["db"] = dz.sum(0)
    return out


def _exact_ids(case, s):
    """The chosen ids by a count of the experts that come before each: those with a larger score,
    or with the same one and a lower id."""
    l = s["logits"].double()
    p = torch.special.expit(l) if case["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    c = p if s["b"] is None else p + s["b"].double()
    n, E, G = c.shape[0], case["E"], case["groups"]

    def place(v):
        lower = torch.ones(v.shape[1], v.shape[1], dtype=torch.bool, device=v.device).tril(-1)
        parts = [((a[:, None, :] > a[:, :, None]) |
                  ((a[:, None, :] == a[:, :, None]) & lower)).sum(2) for a in v.split(1024)]
        return torch.cat(parts)

    if G > 1:
        best = c.view(n, G, -1).topk(min(case["group_top"], E // G), dim=2).values.sum(2)
        kept = place(best) < case["topk_groups"]
        c = torch.where(kept.repeat_interleave(E // G, 1), c, torch.full_like(c, -math.inf))
    at = place(c)
    return at.argsort(1)[:, :case["topk"]]
