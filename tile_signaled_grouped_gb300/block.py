"""The feed-forward half of a transformer block around the routed experts.

    s = x + residual,  h = layer norm of s
    ids, w = the router's choice from the scores h W_router^T
    moe = the routed experts' weighted outputs for h          (runtime.ExpertCombine)
    y = act(h W1^T + b1) W2^T + b2 + s                        (a dense expert for every token)

and, for training, the backward pass of everything but the routed experts' weights.
Argument checks and output allocation are those of ops and runtime, and the computation
their kernels; only gradients that meet are added by torch, in their own 16 bits (a rounding each).
"""
from __future__ import annotations

import torch

from . import ops
from .runtime import ExpertCombine


class MoEBlock:
    """One block's feed-forward half, its tokens split over the layer's W logical ranks.

    layer: an ExpertCombine; router: an ops.router_cfg with its E and topk. Parameters, on
    the layer's device: norm_w, norm_b [D]; w_router [E, D]; router_bias [E] fp32 or None;
    w1 [H, D], b1 [H]; w2 [D, H], b2 [D] (biases may be None); w_gate, w_up, w_down: the
    routed experts' weights as ExpertCombine takes them. Matrices are bf16."""

    def __init__(self, layer: ExpertCombine, router, norm_w, norm_b, w_router, w1, b1, w2, b2,
                 w_gate, w_up, w_down, router_bias=None, act="silu", eps=1e-5):
        self.layer, self.router, self.router_bias = layer, router, router_bias
        self.norm_w, self.norm_b, self.eps = norm_w, norm_b, eps
        self.w_router, self.w1, self.b1, self.w2, self.b2 = w_router, w1, b1, w2, b2
        self.w_gate, self.w_up, self.w_down, self.act = w_gate, w_up, w_down, act
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
                         ids=lay.ids.view(n, -1).clone())
        return y, moe, saved

    def backward(self, dy, saved, d_w=None, dh=None):
        """Gradients of forward() from dy, the gradient of y: a dict with x (which is the
        residual's too), norm_w, norm_b, w1, b1, w2, b2 and, given d_w [W*T, topk] fp32 (the
        gradient of the routing weights), w_router. The routed experts are not trained here;
        dh, the gradient of h through them, is added if given."""
        g = {}
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
