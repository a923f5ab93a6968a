"""The operators of a transformer block around the routed experts, on torch tensors.

route_experts, layer_norm and linear with their backward passes: argument checks and
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
    gradient too), for its x, weight, act and the z that it returned with preact.

    bias: the type of dbias (x's or torch.float32), or None for no dbias. dweight has
    dw_dtype (x's type or fp32; default x's). The products take dy act'(z) rounded to x's
    type."""
    if stream is not None:
        with _on(x, stream):
            return linear_backward(dy, x, weight, z, act, bias, dw_dtype, need_dx, need_dw)
    return (_native or native()).linear_backward(dy, x, weight, z, act, bias, dw_dtype, need_dx,
                                                 need_dw)


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
