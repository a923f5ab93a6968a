"""The operators that train and serve the routed experts of a transformer block on any batch, as cases to
measure: tokens to rows sorted by expert and back, the experts' products, their gated activation, and
activations kept in 8 bits for the backward pass.

A case is a dict of plain values; "op" says which operator and direction:
  dispatch       the order of the tokens' slots by expert, and the tokens as rows in that order
  dispatch_grad  the gradient of the tokens from that of the rows
  combine        y = sum over a token's slots of weight times row
  combine_grad   the gradients of the rows and of the weights
  experts        y = W[e] x for the rows of every expert e
  experts_grad   the gradients of x and of every W[e]
  gated          h = act(gate) up, and its gradients from what was kept of gate and up
  checkpoint     a matrix to 8 bits and back
  linear_grad    the gradients of a dense product whose activations were kept in 8 bits

An 8-bit checkpoint holds a row in blocks of 32 elements: a power of two 2^s, the least for which
the block's largest element is at most 448 2^s, and e4m3 codes of the elements over it.

With own = False, run() computes them in elementary torch operations; with own = True it calls
tile_signaled_grouped_gb300.ops. exact() computes them in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 32  # elements that share a scale


def _rows(name, op, T, E, topk, D, dtype, pad=0, drop=False, eight=False):
    return dict(name=name, op=op, T=T, E=E, topk=topk, D=D, dtype=dtype, pad=pad, drop=drop,
                eight=eight)


def _experts(name, op, T, E, topk, N, K, dtype, pad=0, drop=False, add=False, dwtype=None):
    return dict(name=name, op=op, T=T, E=E, topk=topk, N=N, K=K, dtype=dtype, pad=pad, drop=drop,
                add=add, dwtype=dwtype or dtype)


def _gated(name, n, F, dtype, act="silu", pad=0, eight=True):
    return dict(name=name, op="gated", n=n, F=F, dtype=dtype, act=act, pad=pad, eight=eight)


def listed():
    return [
        # One token of a decoding step to the rows of its 8 experts: latency.
        _rows("dispatch one token", "dispatch", 1, 256, 8, 7168, "bf16"),
        # A training batch or prompt to expert rows: each token is read once and written 8 times.
        _rows("dispatch prompt", "dispatch", 8192, 128, 8, 4096, "bf16"),
        # An odd batch back from rows of an odd length inside wider ones; some slots have no expert.
        _rows("combine ragged", "combine", 1001, 120, 6, 1531, "fp16", pad=5, drop=True),
        # The backward pass of that sum over a training batch, the experts' rows kept in 8 bits.
        _rows("combine gradient", "combine_grad", 4096, 256, 8, 7168, "bf16", eight=True),
        # One token through a matrix of its 8 experts: reads their weights once.
        _experts("experts one token", "experts", 1, 64, 8, 2048, 7168, "bf16"),
        # An odd batch over many small experts, some of them without a row.
        _experts("experts ragged", "experts", 777, 60, 6, 1000, 1544, "fp16", pad=8, drop=True),
        # A prompt or training batch through a matrix of 128 experts of uneven load.
        _experts("experts prompt", "experts", 4096, 128, 8, 2048, 4096, "bf16"),
        # The backward pass of the large matrices of 8 experts.
        _experts("experts gradient", "experts_grad", 4096, 8, 2, 8192, 2048, "bf16"),
        # A training step's gated activation: forward, and backward from 8 bits.
        _gated("gated batch", 32768, 2048, "bf16"),
        # Odd rows of an odd length inside wider rows, kept as they are.
        _gated("gated ragged", 1333, 1531, "fp16", act="gelu", pad=5, eight=False),
        # A batch's hidden states to 8 bits and back.
        dict(name="checkpoint batch", op="checkpoint", n=8192, D=7168, dtype="bf16", pad=0),
        # The backward pass of a dense expert's matrix whose input and product were kept in 8 bits.
        dict(name="linear gradient from 8 bits", op="linear_grad", M=8192, N=2048, K=4096, dtype="bf16",
             act="silu", bias=True, pad=0),
    ]


def _count(rng, most):
    """1 to `most`, even in the logarithm: a power of two, or an odd number."""
    v = min(math.exp(rng.uniform(0.0, math.log(most + 1))), most)
    return 1 << int(math.log2(v)) if rng.random() < 0.4 else max(1, int(v) - 1 + int(v) % 2)


def draw(rng):
    """A case of the ranges that the listed ones stand for: any operator, from one token on."""
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "experts", "experts",
                     "experts_grad", "experts_grad", "gated", "checkpoint", "linear_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    E = rng.choice([8, 16, 64, 128, 256, rng.randint(2, 255)])
    topk = rng.randint(1, min(8, E))
    pad = rng.choice([0, 0, 5, 8])
    drop = rng.random() < 0.3
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        if op != "combine_grad" and rng.random() < 0.2:
            dtype = "fp32"
        D = rng.choice([128, 1536, 2048, 4096, 5120, 7168, 2 * rng.randint(20, 3583) + 1])
        return dict(op=op, T=_count(rng, min(16384, (1 << 27) // (D * topk))), E=E, topk=topk, D=D,
                    dtype=dtype, pad=pad, drop=drop, eight=op == "combine_grad" and rng.random() < 0.5)
    if op in ("experts", "experts_grad"):
        N = rng.choice([128, 256, 1536, 2048, 4096, 8192, 8 * (2 * rng.randint(1, 400) + 1)])
        K = rng.choice([128, 256, 1536, 2048, 4096, 7168, 8 * (2 * rng.randint(1, 400) + 1)])
        E = min(E, max(2, (1 << 30) // (N * K)))
        topk = min(topk, E)
        most = min(16384, (1 << (37 if op == "experts_grad" else 38)) // (N * K * topk))
        return dict(op=op, T=_count(rng, most), E=E, topk=topk, N=N, K=K, dtype=dtype,
                    pad=rng.choice([0, 0, 8]), drop=drop,
                    add=op == "experts_grad" and rng.random() < 0.5,
                    dwtype=rng.choice([dtype, "fp32"]))
    if op == "gated":
        F = rng.choice([128, 1536, 2048, 8192, 2 * rng.randint(20, 4095) + 1])
        return dict(op=op, n=_count(rng, (1 << 26) // F), F=F, dtype=dtype,
                    act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]), pad=pad,
                    eight=rng.random() < 0.6)
    if op == "checkpoint":
        D = rng.choice([128, 1536, 2048, 4096, 5120, 7168, 2 * rng.randint(20, 3583) + 1])
        return dict(op=op, n=_count(rng, (1 << 26) // D), D=D,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), pad=pad)
    N = rng.choice([128, 256, 1536, 2048, 4096, 8 * (2 * rng.randint(1, 255) + 1)])
    K = rng.choice([128, 256, 1536, 2048, 4096, 7168, 8 * (2 * rng.randint(1, 511) + 1)])
    return dict(op=op, M=_count(rng, min(8192, (1 << 36) // (N * K))), N=N, K=K, dtype=dtype,
                act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.8,
                pad=rng.choice([0, 0, 8]))


# ------------------------------------------------------------------------------------- inputs
class _Maker:
    """Seeded tensors on the GPU."""

    def __init__(self, seed):
        self.dev = "cuda" if torch.cuda.is_available() else "cpu"
        self.g = torch.Generator(device=self.dev)
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, device=self.dev, dtype=dtype).normal_(0.0, std, generator=self.g)

    def uniform(self, *shape):
        return torch.rand(shape, device=self.dev, generator=self.g)

    def rows(self, n, c, dtype, pad, std=1.0):
        """n rows of c elements, as the first columns of rows that are `pad` elements wider."""
        t = torch.zeros(n, c + pad, dtype=dtype, device=self.dev)
        t[:, :c] = self.normal(n, c, std=std)
        return t[:, :c]

    def hidden(self, n, c, dtype, pad):
        """Rows whose channels differ in size, as hidden states have them."""
        t = self.rows(n, c, dtype, pad)
        t.mul_(torch.exp(self.normal(c, std=0.5)).to(dtype))
        return t


def _ids(mk, T, E, topk, drop):
    """Distinct experts of every token, some of them chosen more often than others; with `drop`
    a tenth of the slots and all of some tokens' have none (-1)."""
    ids = (mk.normal(T, E) + mk.normal(E, std=0.5)).topk(topk, dim=1).indices.to(torch.int32)
    if drop:
        ids.masked_fill_(mk.uniform(T, topk) < 0.1, -1)
        ids[mk.uniform(T) < 0.02] = -1
    return ids


def _order(ids, E):
    """(slots, rows, offsets): the slots t * topk + j in the order of their experts (-1 behind
    the last), the row of each slot (-1: none), and every expert's first row."""
    n = ids.numel()
    key = ids.reshape(-1)
    key = torch.where((key >= 0) & (key < E), key, torch.full_like(key, E))
    s, at = key.sort(stable=True)
    offsets = torch.searchsorted(s, torch.arange(E + 1, device=key.device, dtype=key.dtype))
    number = torch.arange(n, device=key.device)
    used = number < offsets[E]
    slots = torch.where(used, at, torch.full_like(at, -1))
    rows = torch.empty_like(at).scatter_(0, at, torch.where(used, number, torch.full_like(at, -1)))
    return slots.to(torch.int32), rows.view(ids.shape).to(torch.int32), offsets.to(torch.int32)


def _to_8_bits(x):
    """(codes, scales): e4m3 codes of x over 2^(scale - 127), a scale for each 32 elements of a row."""
    n, c = x.shape
    blocks = (c + BLOCK - 1) // BLOCK
    v = torch.zeros(n, blocks * BLOCK, device=x.device)
    v[:, :c] = x.float()
    v = v.view(n, blocks, BLOCK)
    m, e = torch.frexp(v.abs().amax(2))  # the largest is m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    s = torch.where(m == 0, torch.full_like(e, -127), torch.where(m <= 0.875, e - 9, e - 8).clamp(-127, 127))
    q = torch.ldexp(torch.ldexp(v, -(s // 2)[:, :, None]), -(s - s // 2)[:, :, None])
    step = torch.exp2((torch.frexp(q).exponent - 1).clamp(min=-6).float() - 3.0)
    q = torch.round(q / step) * step  # to nearest, ties to even
    codes = q.view(n, -1)[:, :c].to(torch.float8_e4m3fn).contiguous()
    return codes, (s + 127).to(torch.uint8)


def _from_8_bits(codes, scales):
    n, c = codes.shape
    f = torch.exp2(scales.double() - 127.0).float()
    return codes.float() * f.repeat_interleave(BLOCK, 1)[:, :c]


def _inputs(case, seed):
    mk = _Maker(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    pad = case["pad"]
    s = dict(case)
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        T, E, topk, D = case["T"], case["E"], case["topk"], case["D"]
        s["ids"] = _ids(mk, T, E, topk, case["drop"])
        if op == "dispatch":
            s["x"] = mk.hidden(T, D, dt, pad)
            return s
        s["order"] = _order(s["ids"], E)  # kept by the forward pass
        s["w"] = mk.uniform(T, topk) * 0.4
        if op == "combine_grad":
            s["dy"] = mk.rows(T, D, dt, pad)
        if case["eight"]:
            s["r8"] = _to_8_bits(mk.hidden(T * topk, D, dt, 0))
        else:
            s["r"] = mk.hidden(T * topk, D, dt, pad)
        return s
    if op in ("experts", "experts_grad"):
        T, E, topk, N, K = case["T"], case["E"], case["topk"], case["N"], case["K"]
        s["order"] = _order(_ids(mk, T, E, topk, case["drop"]), E)
        s["starts"] = s["order"][2].tolist()
        s["x"] = mk.rows(T * topk, K, dt, pad)
        s["weight"] = mk.normal(E, N, K, std=1.0 / math.sqrt(K), dtype=dt)
        if op == "experts_grad":
            s["dy"] = mk.rows(T * topk, N, dt, pad)
            s["prior"] = mk.rows(T * topk, K, dt, pad) if case["add"] else None
        return s
    if op == "gated":
        for name in ("gate", "up", "dh"):
            s[name] = mk.rows(case["n"], case["F"], dt, pad, std=1.5 if name == "gate" else 1.0)
        return s
    if op == "checkpoint":
        s["x"] = mk.hidden(case["n"], case["D"], dt, pad)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s["x8"] = _to_8_bits(mk.hidden(M, K, dt, 0))  # kept by the forward pass
    s["z8"] = _to_8_bits(mk.rows(M, N, dt, 0)) if case["act"] != "none" else None
    s["weight"] = mk.rows(N, K, dt, pad, std=1.0 / math.sqrt(K))
    s["dy"] = mk.rows(M, N, dt, pad)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---------------------------------------------------------------------------------- plain form
def _taken(r, rows):
    """The rows r[rows] in 32 bits, zeros where there is none: [T, topk, D]."""
    got = r[rows.long().clamp(min=0)].float()
    return torch.where(rows[:, :, None] >= 0, got, torch.zeros_like(got))


def _row_tokens(slots, topk):
    """The token of every row (0 where the row has none), and which rows have one."""
    return slots.long().clamp(min=0) // topk, slots >= 0


def _dispatch_plain(s):
    slots, rows, offsets = _order(s["ids"], s["E"])
    at, used = _row_tokens(slots, s["topk"])
    x = s["x"][at]
    return {"slots": slots, "rows": rows, "offsets": offsets,
            "x": torch.where(used[:, None], x, torch.zeros_like(x))}


def _dispatch_grad_plain(s):
    return {"dx": _taken(s["r"], s["order"][1]).sum(1).to(s["r"].dtype)}


def _combine_plain(s):
    return {"y": (_taken(s["r"], s["order"][1]) * s["w"][:, :, None]).sum(1).to(s["r"].dtype)}


def _combine_grad_plain(s):
    slots, rows, _ = s["order"]
    r = _from_8_bits(*s["r8"]) if s["eight"] else s["r"]
    dy = s["dy"].float()
    dw = torch.stack([(_taken(r, rows[:, j:j + 1])[:, 0] * dy).sum(1) for j in range(s["topk"])], 1)
    at, used = _row_tokens(slots, s["topk"])
    w = torch.where(used, s["w"].view(-1)[slots.long().clamp(min=0)], torch.zeros_like(s["w"].view(-1)))
    dr = torch.where(used[:, None], dy[at] * w[:, None], torch.zeros((), device=dy.device))
    return {"dr": dr.to(s["dy"].dtype), "dw": dw}


def _experts_plain(s):
    x, w, starts = s["x"], s["weight"], s["starts"]
    y = torch.zeros(x.shape[0], s["N"], dtype=x.dtype, device=x.device)
    for e in range(s["E"]):
        a, b = starts[e], starts[e + 1]
        if b > a:
            y[a:b] = x[a:b].float() @ w[e].float().t()
    return {"y": y}


def _experts_grad_plain(s):
    x, w, dy, starts = s["x"], s["weight"], s["dy"], s["starts"]
    dx = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
    dw = torch.zeros(w.shape, dtype=TYPES[s["dwtype"]], device=x.device)
    for e in range(s["E"]):
        a, b = starts[e], starts[e + 1]
        if b > a:
            d = dy[a:b].float() @ w[e].float()
            dx[a:b] = d + s["prior"][a:b].float() if s["add"] else d
            dw[e] = dy[a:b].float().t() @ x[a:b].float()
    if s["add"]:
        dx[starts[-1]:] = s["prior"][starts[-1]:]
    return {"dx": dx, "dw": dw}


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


def _gated_plain(s):
    g, u, act, dt = s["gate"], s["up"], s["act"], s["gate"].dtype
    out = {"h": (_act(g.float(), act) * u.float()).to(dt)}
    if s["eight"]:
        g, u = _from_8_bits(*_to_8_bits(g)), _from_8_bits(*_to_8_bits(u))
    g, u, dh = g.float(), u.float(), s["dh"].float()
    a = _act(g, act)
    out.update(d_gate=(dh * u * _act_grad(g, act)).to(dt), d_up=(dh * a).to(dt), again=(a * u).to(dt))
    return out


def _checkpoint_plain(s):
    return {"x": _from_8_bits(*_to_8_bits(s["x"])).to(s["x"].dtype)}


def _linear_grad_plain(s):
    dt, dz = s["dy"].dtype, s["dy"].float()
    if s["z8"] is not None:
        dz = dz * _act_grad(_from_8_bits(*s["z8"]), s["act"])
    out = {"dx": (dz @ s["weight"].float()).to(dt), "dw": (dz.t() @ _from_8_bits(*s["x8"])).to(dt)}
    if s["bias"]:
        out["db"] = dz.sum(0)
    return out


# ------------------------------------------------------------------------------- the framework
def _run_own(s):
    from tile_signaled_grouped_gb300 import ops

    op = s["op"]
    if op == "dispatch":
        order = ops.sort_experts(s["ids"], s["E"])
        return {"slots": order.slots, "rows": order.rows, "offsets": order.offsets,
                "x": ops.expert_rows(s["x"], order)}
    if op == "dispatch_grad":
        return {"dx": ops.expert_rows_backward(s["r"], ops.ExpertOrder(*s["order"]))}
    if op == "combine":
        return {"y": ops.combine_experts(s["r"], s["w"], ops.ExpertOrder(*s["order"]))}
    if op == "combine_grad":
        r = ops.Checkpoint(*s["r8"]) if s["eight"] else s["r"]
        dr, dw = ops.combine_experts_backward(s["dy"], r, s["w"], ops.ExpertOrder(*s["order"]))
        return {"dr": dr, "dw": dw}
    if op == "experts":
        return {"y": ops.expert_linear(s["x"], s["weight"], s["order"][2])}
    if op == "experts_grad":
        dx, dw = ops.expert_linear_backward(s["dy"], s["x"], s["weight"], s["order"][2], add=s["prior"],
                                            dw_dtype=TYPES[s["dwtype"]])
        return {"dx": dx, "dw": dw}
    if op == "gated":
        h, saved = ops.gated(s["gate"], s["up"], act=s["act"], checkpoint=s["eight"])
        gate, up = saved if s["eight"] else (s["gate"], s["up"])
        d_gate, d_up, again = ops.gated_backward(s["dh"], gate, up, act=s["act"], need_h=True)
        return {"h": h, "d_gate": d_gate, "d_up": d_up, "again": again}
    if op == "checkpoint":
        return {"x": ops.restore(ops.checkpoint(s["x"]), s["x"].dtype)}
    dx, dw, db = ops.linear_backward(s["dy"], ops.Checkpoint(*s["x8"]), s["weight"],
                                     z=None if s["z8"] is None else ops.Checkpoint(*s["z8"]),
                                     act=s["act"], bias=torch.float32 if s["bias"] else None)
    return {"dx": dx, "dw": dw, "db": db} if s["bias"] else {"dx": dx, "dw": dw}


def run(state):
    if own:
        return _run_own(state)
    return {"dispatch": _dispatch_plain, "dispatch_grad": _dispatch_grad_plain,
            "combine": _combine_plain, "combine_grad": _combine_grad_plain,
            "experts": _experts_plain, "experts_grad": _experts_grad_plain, "gated": _gated_plain,
            "checkpoint": _checkpoint_plain, "linear_grad": _linear_grad_plain}[state["op"]](state)


def _in_8_bits(n, c):
    return n * (c + (c + BLOCK - 1) // BLOCK)


def work(case):
    """Each input read once and each output written once; the operations of the products, and of
    the elementwise parts a handful for each element. Of the experts' weights those that the
    expected number of experts with rows have."""
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        T, n, D = case["T"], case["T"] * case["topk"], case["D"]
        if op == "dispatch":
            return {"bytes": (T + n) * D * e + 12 * n + 4 * case["E"], "flops": 10 * n}
        if op == "combine_grad":
            r = _in_8_bits(n, D) if case["eight"] else n * D * e
            return {"bytes": (T + n) * D * e + r + 12 * n, "flops": 3 * n * D}
        return {"bytes": (T + n) * D * e + (4 if op == "dispatch_grad" else 8) * n, "flops": 2 * n * D}
    if op in ("experts", "experts_grad"):
        n, E, N, K = case["T"] * case["topk"], case["E"], case["N"], case["K"]
        live = E * (1.0 - (1.0 - case["topk"] / E) ** case["T"])
        if op == "experts":
            return {"bytes": int(live * N * K * e) + n * (N + K) * e, "flops": 2 * n * N * K}
        rows = n * (N + (3 if case["add"] else 2) * K) * e
        return {"bytes": int(live * N * K * e) + E * N * K * BYTES[case["dwtype"]] + rows,
                "flops": 4 * n * N * K}
    if op == "gated":
        n, F = case["n"], case["F"]
        kept = 4 * _in_8_bits(n, F) if case["eight"] else 2 * n * F * e
        return {"bytes": 7 * n * F * e + kept, "flops": 30 * n * F}
    if op == "checkpoint":
        n, D = case["n"], case["D"]
        return {"bytes": 2 * n * D * e + 2 * _in_8_bits(n, D), "flops": 4 * n * D}
    M, N, K = case["M"], case["N"], case["K"]
    kept = _in_8_bits(M, K) + (_in_8_bits(M, N) if case["act"] != "none" else 0)
    return {"bytes": kept + e * (M * N + M * K + 2 * N * K) + (4 * N if case["bias"] else 0),
            "flops": 4 * M * N * K}


# ------------------------------------------------------------------------------ 64-bit results
def _exact_order(ids, E):
    """The order by counting: a slot's row is the slots of lower experts and the earlier ones of its own."""
    T, topk = ids.shape
    n = T * topk
    flat = ids.reshape(-1).long()
    of = torch.zeros(n, E, dtype=torch.int32, device=ids.device)
    kept = torch.nonzero((flat >= 0) & (flat < E))[:, 0]
    of[kept, flat[kept]] = 1
    counts = of.sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = counts.cumsum(0)
    earlier = of.cumsum(0)
    rows = torch.full((n,), -1, dtype=torch.int64, device=ids.device)
    rows[kept] = offsets[flat[kept]] + earlier[kept, flat[kept]] - 1
    slots = torch.full((n,), -1, dtype=torch.int64, device=ids.device)
    slots[rows[kept]] = kept
    return slots, rows.view(T, topk), offsets


def _exact_8_bits(x):
    """What an 8-bit checkpoint of x stands for, in 64 bits, from the table of the e4m3 numbers."""
    table = [m * 2.0 ** -9 for m in range(8)]
    table += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    t = torch.tensor(table[:127], dtype=torch.float64, device=x.device)  # the last is 448
    n, c = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -c % BLOCK)).view(n, -1, BLOCK)
    largest = v.abs().amax(2, keepdim=True)
    # (Elements of 32 bits and fewer: past a power of two, the logarithm is past it by 8e-8 at least.)
    s = torch.ceil(torch.log2(largest / 448.0) - 1e-9).clamp(-127, 127)
    unit = torch.exp2(torch.where(largest > 0, s, torch.full_like(s, -127.0)))
    a = v.abs() / unit
    hi = torch.searchsorted(t, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = t[hi] - a, a - t[lo]
    at = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (torch.sign(v) * t[at] * unit).view(n, -1)[:, :c]


def _act64(act):
    F = torch.nn.functional
    return {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[act]


def _decoded(kept):
    codes, scales = kept
    f = torch.ldexp(torch.ones(scales.shape, dtype=torch.float64, device=codes.device), scales.int() - 127)
    return codes.double() * f.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "dispatch":
        slots, rows, offsets = _exact_order(s["ids"], case["E"])
        x = torch.zeros(slots.numel(), case["D"], dtype=torch.float64, device=slots.device)
        for j in range(case["topk"]):
            used = rows[:, j] >= 0
            x[rows[used, j]] = s["x"][used].double()
        return {"slots": slots.int(), "rows": rows.int(), "offsets": offsets.int(), "x": x}
    if op in ("dispatch_grad", "combine", "combine_grad"):
        T, topk, D = case["T"], case["topk"], case["D"]
        rows = s["order"][1].long()
        n = T * topk
        r = _decoded(s["r8"]) if case["eight"] else s["r"]
        w = s["w"].double()
        y = torch.zeros(T, D, dtype=torch.float64, device=w.device)
        dr = torch.zeros(n if op == "combine_grad" else 0, D, dtype=torch.float64, device=w.device)
        dw = torch.zeros(T, topk, dtype=torch.float64, device=w.device)
        for j in range(topk):
            t = torch.nonzero(rows[:, j] >= 0)[:, 0]
            at = rows[t, j]
            got = r[at].double()
            if op == "combine_grad":
                d = s["dy"][t].double()
                dr[at] = w[t, j, None] * d
                dw[t, j] = torch.einsum("td,td->t", d, got)
            else:
                y[t] += got if op == "dispatch_grad" else w[t, j, None] * got
        return {"dr": dr, "dw": dw} if op == "combine_grad" else {"dx" if op == "dispatch_grad" else "y": y}
    if op in ("experts", "experts_grad"):
        x, weight, offsets = s["x"], s["weight"], s["order"][2].long().tolist()
        y = torch.zeros(x.shape[0], case["N"] if op == "experts" else case["K"], dtype=torch.float64,
                        device=x.device)
        dw = torch.zeros(weight.shape if op == "experts_grad" else (0,), dtype=torch.float64,
                         device=x.device)
        if op == "experts_grad" and s["prior"] is not None:
            y += s["prior"].double()
        for e, w in enumerate(weight):
            at = slice(offsets[e], offsets[e + 1])
            if op == "experts":
                y[at] = torch.einsum("rk,nk->rn", x[at].double(), w.double())
            else:
                d = s["dy"][at].double()
                y[at] += torch.einsum("rn,nk->rk", d, w.double())
                dw[e] = torch.einsum("rn,rk->nk", d, x[at].double())
        return {"y": y} if op == "experts" else {"dx": y, "dw": dw}
    if op == "gated":
        act, dh = _act64(case["act"]), s["dh"].double()
        g, u = s["gate"].double(), s["up"].double()
        h = act(g) * u
        if case["eight"]:
            g, u = _exact_8_bits(g), _exact_8_bits(u)
        g.requires_grad_()
        u.requires_grad_()
        again = act(g) * u
        d_gate, d_up = torch.autograd.grad(again, (g, u), dh)
        return {"h": h, "d_gate": d_gate, "d_up": d_up, "again": again.detach()}
    if op == "checkpoint":
        return {"x": _exact_8_bits(s["x"])}
    dz, w, x = s["dy"].double(), s["weight"].double(), _decoded(s["x8"])
    if s["z8"] is not None:
        z = _decoded(s["z8"]).requires_grad_()
        (dz,) = torch.autograd.grad(_act64(case["act"])(z), z, dz)
    out = {"dx": torch.einsum("mn,nk->mk", dz, w), "dw": torch.einsum("mn,mk->nk", dz, x)}
    if case["bias"]:
        out["db"] = dz.sum(0)
    return out
