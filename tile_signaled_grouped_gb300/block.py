"""The feed-forward half of a transformer block around the routed experts.

    s = x + residual,  h = layer norm of s
    ids, w = the router's choice from the scores h W_router^T
    moe = the routed experts' weighted outputs for h          (runtime.ExpertCombine)
    y = act(h W1^T + b1) W2^T + b2 + s                        (a dense expert for every token)

and, for training, the backward pass: of everything but the routed experts with the layer, of
these too with Experts, which runs them on rows sorted by expert, for any number of tokens.
Argument checks and output allocation are those of ops and runtime, and the computation
their kernels; only gradients that meet are added by torch, in their own 16 bits (a rounding each).
"""
from __future__ import annotations

import torch

from . import ops
from .runtime import ExpertCombine


class Experts:
    """The routed experts on rows sorted by expert: for every token h and its choices e with weights v,
    y = sum of v * W_down[e] (act(W_gate[e] h) * (W_up[e] h)), and the gradients of it.

    w_gate, w_up [E, F, D], w_down [E, D, F]: bf16 or fp16, D and F multiples of 8. The lists that an
    ExpertCombine of W ranks takes are views of them (ranks()), so both run on the same weights.
    keep: what forward() keeps of a row for backward(), "8 bits" (gate, up and the expert's output as
    ops.Checkpoint: D + 2 F bytes and their 32nd part) or "whole" (twice that). The tokens' rows and
    the product of the gated activation are made again."""

    def __init__(self, w_gate, w_up, w_down, act="silu", keep="8 bits"):
        if keep not in ("8 bits", "whole"):
            raise ValueError(f"keep {keep!r}: expected '8 bits' or 'whole'")
        E, F, D = w_gate.shape
        if w_up.shape != (E, F, D) or w_down.shape != (E, D, F):
            raise ValueError(f"w_gate {tuple(w_gate.shape)}, w_up {tuple(w_up.shape)} and w_down "
                             f"{tuple(w_down.shape)}: expected [E, F, D], [E, F, D] and [E, D, F]")
        self.w_gate, self.w_up, self.w_down, self.act, self.keep = w_gate, w_up, w_down, act, keep

    def ranks(self, W):
        """(w_gate, w_up, w_down) as lists of W ranks' [E / W, ...] views."""
        return tuple(list(w.unflatten(0, (W, -1)).unbind(0)) for w in (self.w_gate, self.w_up, self.w_down))

    def forward(self, h, ids, w, save=False):
        """(y, saved) for h [..., D] and ids, w [..., topk] as ops.route_experts returns them, on the
        current stream. saved (with `save`, else None) is what backward() takes."""
        order = ops.sort_experts(ids, self.w_gate.shape[0])
        x = ops.expert_rows(h, order)
        gate = ops.expert_linear(x, self.w_gate, order.offsets)
        up = ops.expert_linear(x, self.w_up, order.offsets)
        eight = save and self.keep == "8 bits"
        a, kept = ops.gated(gate, up, act=self.act, checkpoint=eight)
        r = ops.expert_linear(a, self.w_down, order.offsets)
        y = ops.combine_experts(r, w, order)
        if not save:
            return y, None
        gate, up = kept if eight else (gate, up)
        return y, dict(h=h, w=w, order=order, gate=gate, up=up, r=ops.checkpoint(r) if eight else r)

    def backward(self, dy, saved):
        """Gradients of forward() from dy, the gradient of y: a dict with h, w, w_gate, w_up and w_down."""
        g, order = {}, saved["order"]
        off = order.offsets
        dr, g["w"] = ops.combine_experts_backward(dy, saved["r"], saved["w"], order)
        da, _ = ops.expert_linear_backward(dr, None, self.w_down, off, need_dw=False)
        d_gate, d_up, a = ops.gated_backward(da, saved["gate"], saved["up"], act=self.act, need_h=True)
        _, g["w_down"] = ops.expert_linear_backward(dr, a, self.w_down, off, need_dx=False)
        x = ops.expert_rows(saved["h"], order)
        dx, g["w_gate"] = ops.expert_linear_backward(d_gate, x, self.w_gate, off)
        dx, g["w_up"] = ops.expert_linear_backward(d_up, x, self.w_up, off, add=dx)
        g["h"] = ops.expert_rows_backward(dx, order)
        return g


class MoEBlock:
    """One block's feed-forward half, its tokens split over the layer's W logical ranks.

    layer: an ExpertCombine; router: an ops.router_cfg with its E and topk. Parameters, on
    the layer's device: norm_w, norm_b [D]; w_router [E, D]; router_bias [E] fp32 or None;
    w1 [H, D], b1 [H]; w2 [D, H], b2 [D] (biases may be None); w_gate, w_up, w_down: the
    routed experts' weights as ExpertCombine takes them. Matrices are bf16. experts: the same weights
    as Experts, to train them: forward() with save then runs them in place of the layer."""

    def __init__(self, layer: ExpertCombine, router, norm_w, norm_b, w_router, w1, b1, w2, b2,
                 w_gate, w_up, w_down, router_bias=None, act="silu", eps=1e-5, experts=None):
        self.layer, self.router, self.router_bias = layer, router, router_bias
        self.norm_w, self.norm_b, self.eps = norm_w, norm_b, eps
        self.w_router, self.w1, self.b1, self.w2, self.b2 = w_router, w1, b1, w2, b2
        self.w_gate, self.w_up, self.w_down, self.act = w_gate, w_up, w_down, act
        self.experts = experts
        self.consumer = torch.cuda.Stream(device=layer.device, priority=-1)

    def forward(self, x, residual=None, save=False):
        """(y, moe, saved) for x [W*T, D] bf16 (rank s's tokens are rows s*T to s*T + T - 1), on
        the current stream. The block's output is y + moe: the next block's norm adds them
        (`residual`), so the sum is not written here. saved (with `save`, else None) is what
        backward() takes."""
        lay = self.layer
        n, d = lay.W * lay.T, lay.D
        if x.shape != (n, d) or not x.is_contiguous():
            raise ValueError(f"x must be contiguous {(n, d)}, got {tuple(x.shape)}")
        h, s, mean, rstd = ops.layer_norm(x, self.norm_w, self.norm_b, eps=self.eps,
                                          residual=residual, stats=save)
        logits, _ = ops.linear(h, self.w_router, out_dtype=torch.float32)
        stream = torch.cuda.current_stream(lay.device)
        lay.route_experts(logits, self.router, bias=self.router_bias, stream=stream)
        routed = None
        if save and self.experts is not None:
            # The layer's ids and weights are those of its last routing: what is kept is a copy.
            ids, w = lay.ids.view(n, -1).clone(), lay.w.view(n, -1).clone()
            moe, routed = self.experts.forward(h, ids, w, save=True)
        else:
            ranks = list(h.view(lay.W, lay.T, d).unbind(0))
            moe = torch.empty_like(h)
            lay.plan_build(ranks, stream=stream)
            lay.expert_combine(self.w_gate, self.w_up, self.w_down, producer=stream,
                               consumer=self.consumer)
            lay.scale_step(stream=stream, out=list(moe.view(lay.W, lay.T, d).unbind(0)))
        a, z = ops.linear(h, self.w1, self.b1, act=self.act, preact=save)
        y, _ = ops.linear(a, self.w2, self.b2, residual=s)
        saved = None
        if save:
            saved = dict(h=h, s=s, mean=mean, rstd=rstd, logits=logits, z=z, a=a,
                         ids=lay.ids.view(n, -1).clone(), routed=routed)
        return y, moe, saved

    def backward(self, dy, saved, d_w=None, dh=None, d_moe=None):
        """Gradients of forward() from dy, the gradient of y: a dict with x (which is the
        residual's too), norm_w, norm_b, w1, b1, w2, b2 and, given d_w [W*T, topk] fp32 (the
        gradient of the routing weights), w_router. The routed experts are trained with Experts
        alone: given d_moe, the gradient of moe, the dict has w_gate, w_up, w_down and w_router too.
        dh, a gradient of h from elsewhere, is added if given."""
        g = {}
        if d_moe is not None:
            if saved["routed"] is None:
                raise ValueError("d_moe is the gradient through Experts, which this block was not given")
            routed = self.experts.backward(d_moe, saved["routed"])
            d_w = routed.pop("w") if d_w is None else d_w + routed.pop("w")
            dh = routed.pop("h") if dh is None else dh + routed.pop("h")
            g.update(routed)
        da, g["w2"], g["b2"] = ops.linear_backward(dy, saved["a"], self.w2, bias=_type(self.b2))
        d_h, g["w1"], g["b1"] = ops.linear_backward(da, saved["h"], self.w1, z=saved["z"],
                                                    act=self.act, bias=_type(self.b1))
        if dh is not None:
            d_h = d_h + dh
        if d_w is not None:
            c = self.router
            dl = ops.route_experts_backward(d_w, saved["logits"], saved["ids"],
                                            score=ops.score_name(c), renorm=bool(c.renorm),
                                            scale=c.scale)
            # The products take 16-bit operands: the scores' gradient is rounded once, as dz is.
            dx, g["w_router"], _ = ops.linear_backward(dl.to(dy.dtype), saved["h"], self.w_router)
            d_h = d_h + dx
        # s is the residual of the second product: its gradient dy joins the norm's.
        g["x"], g["norm_w"], g["norm_b"] = ops.layer_norm_backward(
            d_h, saved["s"], self.norm_w, saved["mean"], saved["rstd"], dz=dy,
            bias=self.norm_b is not None)
        return g


def _type(bias):
    return None if bias is None else bias.dtype
