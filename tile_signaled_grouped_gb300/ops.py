"""The operators of a transformer block around and inside the routed experts, on torch tensors.

route_experts, layer_norm and linear, the way to the experts' rows and back (sort_experts, expert_rows,
combine_experts), the experts' products (expert_linear) and their activation (gated), with their
backward passes, and activations kept in 8 bits (checkpoint, restore): argument checks and
output allocation over the C ABI, in csrc/torch_ops.cpp; every computation is a launch of
the library's kernels. A matrix is a tensor whose last dimension is contiguous and whose
other dimensions are one run of rows (any 2-D tensor with a row stride; more dimensions
as `view` can join them).

They are not known to autograd: tensors that require a gradient are taken as their values,
results carry no history, and a backward pass is the call that bears its name.

Every call is asynchronous on `stream` (default: the current one) and may be captured
into a CUDA graph after a first call. Outputs are allocated on that stream. Inputs
written on another stream must be complete before it (an event or a synchronize) and
stay alive until the call has run there.
"""
from __future__ import annotations

import contextlib
import os
from typing import NamedTuple

import torch

from . import build, capi
from .runtime import _stream_handle

_SCORES = {"softmax": capi.MOE_SCORE_SOFTMAX, "sigmoid": capi.MOE_SCORE_SIGMOID}
_native = None


def native():
    """The module of csrc/torch_ops.cpp: the checks, allocations and C calls of this file's
    functions."""
    global _native
    if _native is None:
        if not os.path.exists(os.path.join(os.path.dirname(capi.LIB_PATH), "_torch_ops.so")):
            why = build.binding_lacks()
            raise capi.MoeError("_torch_ops.so is missing: the torch binding is not built (run "
                                "tile_signaled_grouped_gb300.build.build()"
                                + (f"; here {why})" if why else ")"))
        from . import _torch_ops

        _torch_ops.set_error(capi.MoeError)
        _native = _torch_ops
    return _native


@contextlib.contextmanager
def _on(t, stream):
    """Makes t's device and `stream` (a torch stream or a raw handle) current: outputs and
    workspaces are then allocated for that stream."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    if stream.device != t.device:
        raise ValueError(f"stream of {stream.device} for tensors of {t.device}")
    with torch.cuda.device(t.device), torch.cuda.stream(stream):
        yield


# ------------------------------------------------------------------------------ routing
def router_cfg(E, topk, score="softmax", groups=1, topk_groups=1, group_top=1, renorm=False,
               scale=1.0) -> capi.moe_router_cfg:
    """The C configuration of a router; its limits are checked by the call that takes it."""
    if score not in _SCORES:
        raise ValueError(f"score {score!r}: expected one of {', '.join(_SCORES)}")
    return capi.moe_router_cfg(E, topk, _SCORES[score], groups, topk_groups, group_top,
                               int(bool(renorm)), scale)


def score_name(cfg: capi.moe_router_cfg) -> str:
    """The score of a router configuration by its name here."""
    return next(k for k, v in _SCORES.items() if v == cfg.score)


def route_experts(logits, topk, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1,
                  renorm=False, scale=1.0, stream=None):
    """The topk experts of every token and their weights, from scores logits [..., E].

    s = softmax or sigmoid of the logits; c = s + bias; of `groups` groups of consecutive
    experts the topk_groups with the largest sums of their group_top (1 or 2) largest c
    stay, and of their experts the topk with the largest c (equal: lower id). The weights
    are the s of the chosen experts, divided by their sum with renorm, times scale.
    Returns (ids int32 [..., topk], weights fp32 [..., topk]). bias: fp32 [E], used for
    the choice alone. Masked experts have logits of -inf; a token whose chosen experts are
    all masked has weights 0. The choice is that of 64-bit arithmetic; without a bias it goes by
    the logits, which tell scores apart that 64 bits round to the same."""
    if stream is not None:
        with _on(logits, stream):
            return route_experts(logits, topk, score, bias, groups, topk_groups, group_top, renorm,
                                 scale)
    return (_native or native()).route(logits, topk, score, bias, groups, topk_groups, group_top,
                                       renorm, scale)


def route_experts_backward(d_w, logits, ids, score="softmax", renorm=False, scale=1.0, stream=None):
    """The gradient of the logits [..., E], in their type, from the gradient d_w [..., topk]
    of the weights, for the logits and ids of a route_experts call with this score, renorm
    and scale. The choice, and so the bias and the groups, has no gradient."""
    if stream is not None:
        with _on(logits, stream):
            return route_experts_backward(d_w, logits, ids, score, renorm, scale)
    return (_native or native()).route_backward(d_w, logits, ids, score, renorm, scale)


# --------------------------------------------------------------------------- layer norm
def layer_norm(x, weight, bias=None, eps=1e-5, residual=None, stats=False, stream=None):
    """(y, z, mean, rstd): z = x + residual and y = (z - mean) * rstd * weight + bias, with
    the mean and rstd = 1 / sqrt(variance + eps) of each row of z.

    x, residual: [..., D] bf16, fp16 or fp32; weight, bias: [D] of that type or both fp32,
    or None. y and z have x's type and are contiguous; z is x itself without a residual.
    mean and rstd (fp32 [...]) are returned with stats, for layer_norm_backward, else None."""
    if stream is not None:
        with _on(x, stream):
            return layer_norm(x, weight, bias, eps, residual, stats)
    return (_native or native()).layer_norm(x, weight, bias, eps, residual, stats)


def layer_norm_backward(dy, z, weight, mean, rstd, dz=None, bias=True, stream=None):
    """(dx, dweight, dbias) of layer_norm from the gradient dy of y, for the z, mean and
    rstd that it returned. dz: the gradient of z from elsewhere (the residual stream), added
    to dx, which is the gradient of x and of the residual alike. dweight and dbias have the
    weight's type (z's if weight is None, and no dweight then); dbias is None without bias."""
    if stream is not None:
        with _on(z, stream):
            return layer_norm_backward(dy, z, weight, mean, rstd, dz, bias)
    return (_native or native()).layer_norm_backward(dy, z, weight, mean, rstd, dz, bias)


# ------------------------------------------------------------------------------- linear
def linear(x, weight, bias=None, act="none", residual=None, preact=False, out_dtype=None,
           stream=None):
    """(y, z): z = x weight^T + bias, y = act(z) + residual, with fp32 sums.

    x: [..., K], weight: [N, K], both bf16 or both fp16, rows on 16 bytes; bias: [N] of that
    type or fp32; act: "none", "relu", "gelu", "gelu_tanh" or "silu"; residual: [..., N] of
    x's type. y has out_dtype (x's type or fp32; default x's), z (with preact, for
    linear_backward, else None) x's type; both are contiguous."""
    if stream is not None:
        with _on(x, stream):
            return linear(x, weight, bias, act, residual, preact, out_dtype)
    return (_native or native()).linear(x, weight, bias, act, residual, preact, out_dtype)


def linear_backward(dy, x, weight, z=None, act="none", bias=None, dw_dtype=None, need_dx=True,
                    need_dw=True, stream=None):
    """(dx, dweight, dbias) of linear from the gradient dy of y (which is the residual's
    gradient too), for its x, weight, act and the z that it returned with preact. x, z or both may be
    their Checkpoints, that of x where its rows hold a multiple of 8 elements.

    bias: the type of dbias (x's or torch.float32), or None for no dbias. dweight has
    dw_dtype (x's type or fp32; default x's). The products take dy act'(z) rounded to x's
    type. An fp32 dweight loses about 1.2e-9 of its norm for each row that is summed at once (1e-5 for 65536
    rows of 256 x 512); expert_linear_backward's does not."""
    if stream is not None:
        with _on(dy, stream):
            return linear_backward(dy, x, weight, z, act, bias, dw_dtype, need_dx, need_dw)
    x, xs = x if isinstance(x, Checkpoint) else (x, None)
    z, zs = z if isinstance(z, Checkpoint) else (z, None)
    return (_native or native()).linear_backward(dy, x, xs, weight, z, zs, act, bias, dw_dtype, need_dx,
                                                 need_dw)


# -------------------------------------------------------------------------- checkpoints
class Checkpoint(NamedTuple):
    """A tensor [..., c] kept in 8 bits for a backward pass: codes (float8_e4m3fn [..., c]) and
    scales (uint8 [..., ceil(c / 32)]). An element is code * 2^(scale - 127); 32 elements of a row
    share a scale, the least for which the largest of them is at most 448 times it."""
    codes: torch.Tensor
    scales: torch.Tensor


def checkpoint(x, stream=None):
    """x [..., c] (bf16, fp16 or fp32) as a Checkpoint: each element is within 2^-4 of itself, or
    within 2^-10 of its block's scale; what is finite stays so in x's type, what is not becomes NaN."""
    if stream is not None:
        with _on(x, stream):
            return checkpoint(x)
    return Checkpoint(*(_native or native()).checkpoint(x))


def restore(kept, dtype, stream=None):
    """The tensor [..., c] that a Checkpoint stands for, in bf16, fp16 or fp32, contiguous."""
    if stream is not None:
        with _on(kept.codes, stream):
            return restore(kept, dtype)
    return (_native or native()).restore(kept.codes, kept.scales, dtype)


# ----------------------------------------------------------------- rows sorted by expert
class ExpertOrder(NamedTuple):
    """A batch's slots (choice j of token t: t * topk + j) in the order of their experts: slots int32 [n],
    the slot of every row (-1 behind the last row); rows int32 [..., topk], the row of every slot (-1:
    it has none); offsets int32 [E + 1]: expert e has the rows offsets[e] to offsets[e + 1] - 1."""
    slots: torch.Tensor
    rows: torch.Tensor
    offsets: torch.Tensor


def sort_experts(ids, E, stream=None):
    """The ExpertOrder of ids int32 [..., topk] (as route_experts returns them) among E experts, up to
    1024. Earlier slots come first in an expert's rows. A slot whose id is not in 0 .. E - 1 (-1, say)
    has no row."""
    if stream is not None:
        with _on(ids, stream):
            return sort_experts(ids, E)
    return ExpertOrder(*(_native or native()).sort_experts(ids, E))


def expert_rows(x, order, stream=None):
    """The tokens x [..., D] (bf16, fp16 or fp32) as the rows [n, D] of an order, n its number of
    slots: row order.rows[t, j] is token t. Rows behind the last are zero."""
    if stream is not None:
        with _on(x, stream):
            return expert_rows(x, order)
    return (_native or native()).expert_rows(x, order.rows, order.offsets)


def expert_rows_backward(d_rows, order, stream=None):
    """The gradient of expert_rows' x from that of its rows [n, D]: a token's is the sum of its
    rows', added in fp32 and rounded once."""
    return combine_experts(d_rows, None, order, stream)


def combine_experts(r, w, order, stream=None):
    """y [..., D]: y[t] = sum over j of w[t, j] * r[order.rows[t, j]], added in fp32 in the order of j and
    rounded once, for the experts' rows r [n, D] (bf16, fp16 or fp32) and weights w fp32 [..., topk] (None:
    ones). Slots without a row have no part in it."""
    if stream is not None:
        with _on(r, stream):
            return combine_experts(r, w, order)
    return (_native or native()).combine_experts(r, w, order.rows, order.offsets)


def combine_experts_backward(dy, r, w, order, stream=None):
    """(d_r, d_w) of combine_experts from the gradient dy of y, for its r (or the Checkpoint of r), w and
    order. d_r has dy's type, and zeros behind the last row; d_w is fp32, 0 for slots without a row. (Without
    weights, w None there, d_r is expert_rows(dy, order).)"""
    if stream is not None:
        with _on(dy, stream):
            return combine_experts_backward(dy, r, w, order)
    r, scales = r if isinstance(r, Checkpoint) else (r, None)
    return (_native or native()).combine_experts_backward(dy, r, scales, w, order.rows, order.offsets)


# ----------------------------------------------------------------------- expert products
def expert_linear(x, weight, offsets, stream=None):
    """y [n, N]: y[r] = weight[e] x[r] for the rows offsets[e] to offsets[e + 1] - 1 of every expert e, with
    fp32 sums; zeros in the rows before offsets[0] and from offsets[E] on.

    x: [n, K], weight: [E, N, K], both bf16 or both fp16, N and K multiples of 8, rows on 16
    bytes; offsets: int32 [E + 1] on the device, ascending, as sort_experts returns them (or a part of
    them, for the experts that weight then holds)."""
    if stream is not None:
        with _on(x, stream):
            return expert_linear(x, weight, offsets)
    return (_native or native()).expert_linear(x, weight, offsets)


def expert_linear_backward(dy, x, weight, offsets, add=None, dw_dtype=None, need_dx=True, need_dw=True,
                           stream=None):
    """(dx, dweight) of expert_linear from the gradient dy of y, for its x (None without need_dw), weight and
    offsets. add [n, K] of x's type, rows on 16 bytes, is added to dx before it is rounded (the gradient through
    another product of the same x).
    dweight has dw_dtype (x's type or fp32; default x's); it is zero for experts without rows. In fp32 it is
    within 1.2e-6 of its norm up to a million rows of an expert. In 16 bits its fp32 sum loses 1.2e-9 of the
    norm for each row: from some 170000 rows of one expert in fp16, 1.4 million in bf16, take fp32 for accuracy."""
    if stream is not None:
        with _on(dy, stream):
            return expert_linear_backward(dy, x, weight, offsets, add, dw_dtype, need_dx, need_dw)
    return (_native or native()).expert_linear_backward(dy, x, weight, offsets, add, dw_dtype, need_dx,
                                                        need_dw)


# ------------------------------------------------------------------------ gated activation
def gated(gate, up, act="silu", checkpoint=False, stream=None):
    """(h, kept): h = act(gate) * up, for gate and up [..., F] both bf16 or both fp16 (columns of one
    matrix, say); act as in linear. kept (with checkpoint, else None): the Checkpoints of gate and
    up for gated_backward."""
    if stream is not None:
        with _on(gate, stream):
            return gated(gate, up, act, checkpoint)
    h, gc, gs, uc, us = (_native or native()).gated(gate, up, act, checkpoint)
    return h, (Checkpoint(gc, gs), Checkpoint(uc, us)) if checkpoint else None


def gated_backward(dh, gate, up, act="silu", need_h=False, stream=None):
    """(d_gate, d_up, h) of gated from the gradient dh of h, for its gate and up or the Checkpoints of both.
    h, act(gate) * up once more (with need_h, else None), is what the product after it was given,
    or stands for it where gate and up are Checkpoints."""
    if stream is not None:
        with _on(dh, stream):
            return gated_backward(dh, gate, up, act, need_h)
    gate, gs = gate if isinstance(gate, Checkpoint) else (gate, None)
    up, us = up if isinstance(up, Checkpoint) else (up, None)
    return (_native or native()).gated_backward(dh, gate, gs, up, us, act, need_h)


def _device_of(stream):
    """Makes a torch stream's device current (the library finds that of any other handle but a
    default stream's, which says nothing of its device)."""
    device = getattr(stream, "device", None)
    return contextlib.nullcontext() if device is None else torch.cuda.device(device)


def status(stream=None):
    """(code, detail) of the operators' device status: 0, or MOE_DEV_TIMEOUT after a device
    wait ran out, on the device of `stream` (a torch stream or a raw handle; default: the current
    one). Synchronises the stream; clear_status() clears it."""
    with _device_of(stream):
        return capi.moe_ops_status(_stream_handle(stream))


def clear_status(stream=None):
    with _device_of(stream):
        capi.moe_ops_status_clear(_stream_handle(stream))
