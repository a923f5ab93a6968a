"""The operators of a transformer block around the routed experts, on torch tensors.

route_experts, layer_norm and linear with their backward passes: argument checks and
output allocation over the C ABI; every computation is a launch of the library's
kernels. A matrix is a tensor whose last dimension is contiguous and whose other
dimensions are one run of rows (any 2-D tensor with a row stride; more dimensions as
`view` can join them).

Every call is asynchronous on `stream` (default: the current one) and may be captured
into a CUDA graph after a first call. Outputs are allocated on that stream. Inputs
written on another stream must be complete before it (an event or a synchronize) and
stay alive until the call has run there.
"""
from __future__ import annotations

import contextlib
import functools

import torch

from . import capi

_DTYPES = {torch.bfloat16: capi.MOE_BF16, torch.float16: capi.MOE_FP16,
           torch.float32: capi.MOE_FP32}
_ACTS = {"none": capi.MOE_ACT_NONE, "relu": capi.MOE_ACT_RELU, "gelu": capi.MOE_ACT_GELU,
         "gelu_tanh": capi.MOE_ACT_GELU_TANH, "silu": capi.MOE_ACT_SILU}
_FP32 = (torch.float32,)
_HALF = (torch.bfloat16, torch.float16)
_SCORES = {"softmax": capi.MOE_SCORE_SOFTMAX, "sigmoid": capi.MOE_SCORE_SIGMOID}


def _stream_here(t, stream):
    """The raw handle of the current stream if a call on `t` runs there (no other stream is
    asked for and t's device is the current one), else None: the call then enters _on and
    starts again. One integer each from torch's binding: a public Stream object costs more
    than the rest of a call's checks."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"tensors must be on a CUDA device, got {t.device}")
    if stream is None and dev == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(dev)
    return None


@contextlib.contextmanager
def _on(t, stream):
    """Makes t's device, and `stream` (a torch stream or a raw handle) if given, current:
    outputs and workspaces are then allocated for that stream."""
    if stream is not None and not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    if stream is not None and stream.device != t.device:
        raise ValueError(f"stream of {stream.device} for tensors of {t.device}")
    with torch.cuda.device(t.device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _dtype(t, what, allowed=None):
    d = _DTYPES.get(t.dtype)
    if d is None or (allowed is not None and t.dtype not in allowed):
        names = ", ".join(str(a) for a in (allowed or _DTYPES))
        raise ValueError(f"{what} has type {t.dtype}: expected {names}")
    return d


def _rows(t, what, cols=None, dev=None):
    """(rows, cols, leading dimension) of a matrix; `dev`: the device index it has to be on."""
    m = t
    if t.dim() != 2:
        try:
            m = t[None] if t.dim() == 1 else t.view(-1, t.shape[-1]) if t.dim() else None
        except RuntimeError:
            m = None
    n, c = m.shape if m is not None else (0, 0)
    s0, s1 = m.stride() if m is not None else (0, 0)
    if m is None or (c > 1 and s1 != 1) or (n > 1 and s0 < c):
        raise ValueError(f"{what} must be rows of contiguous elements, got shape "
                         f"{tuple(t.shape)} and strides {t.stride()}")
    if cols is not None and c != cols:
        raise ValueError(f"{what} has rows of {c} elements: expected {cols}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}: expected device {dev}")
    return n, c, (s0 if n > 1 else c)


def _vector(t, what, size, dtypes, dev):
    if (t.dim() != 1 or t.shape[0] != size or t.dtype not in dtypes or t.get_device() != dev or
            not t.is_contiguous()):
        raise ValueError(f"{what} must be {size} contiguous elements of "
                         f"{', '.join(str(d) for d in dtypes)} beside the rows, got "
                         f"{tuple(t.shape)} of {t.dtype} on {t.device}")


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------------------ routing
@functools.lru_cache(maxsize=256)
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
    all masked has weights 0. The choice is that of 64-bit arithmetic."""
    n, E, ld = _rows(logits, "logits")
    dt = _dtype(logits, "logits")
    if bias is not None:
        _vector(bias, "bias", E, _FP32, logits.get_device())
    cfg = router_cfg(E, topk, score, groups, topk_groups, group_top, renorm, scale)
    s = _stream_here(logits, stream)
    if s is None:
        with _on(logits, stream):
            return route_experts(logits, topk, score, bias, groups, topk_groups, group_top, renorm,
                                 scale)
    dev = logits.device
    shape = (n, topk) if logits.dim() == 2 else (*logits.shape[:-1], topk)
    ids = torch.empty(shape, dtype=torch.int32, device=dev)
    w = torch.empty(shape, dtype=torch.float32, device=dev)
    capi.moe_router(None, cfg, logits.data_ptr(), dt, n, ld, _ptr(bias), ids.data_ptr(),
                    w.data_ptr(), s)
    return ids, w


def route_experts_backward(d_w, logits, ids, score="softmax", renorm=False, scale=1.0, stream=None):
    """The gradient of the logits [..., E], in their type, from the gradient d_w [..., topk]
    of the weights, for the logits and ids of a route_experts call with this score, renorm
    and scale. The choice, and so the bias and the groups, has no gradient."""
    n, E, ld = _rows(logits, "logits")
    dt = _dtype(logits, "logits")
    for t, what, dtype in ((ids, "ids", torch.int32), (d_w, "d_w", torch.float32)):
        if (t.dtype != dtype or t.shape[:-1] != logits.shape[:-1] or not t.is_contiguous() or
                t.shape[-1:] != ids.shape[-1:] or t.device != logits.device):
            raise ValueError(f"{what} must be contiguous {dtype} of shape [..., topk] beside the "
                             f"logits, got {tuple(t.shape)} of {t.dtype} on {t.device}")
    cfg = router_cfg(E, ids.shape[-1], score, 1, 1, 1, renorm, scale)
    s = _stream_here(logits, stream)
    if s is None:
        with _on(logits, stream):
            return route_experts_backward(d_w, logits, ids, score, renorm, scale)
    d = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    capi.moe_router_backward(cfg, d_w.data_ptr(), logits.data_ptr(), ids.data_ptr(), dt, n, ld,
                             d.data_ptr(), E, s)
    return d


# --------------------------------------------------------------------------- layer norm
def _norm_params(what, t, x, D):
    if t is not None:
        _vector(t, what, D, (x.dtype, torch.float32), x.get_device())


def layer_norm(x, weight, bias=None, eps=1e-5, residual=None, stats=False, stream=None):
    """(y, z, mean, rstd): z = x + residual and y = (z - mean) * rstd * weight + bias, with
    the mean and rstd = 1 / sqrt(variance + eps) of each row of z.

    x, residual: [..., D] bf16, fp16 or fp32; weight, bias: [D] of that type or both fp32,
    or None. y and z have x's type and are contiguous; z is x itself without a residual.
    mean and rstd (fp32 [...]) are returned with stats, for layer_norm_backward, else None."""
    n, D, ld = _rows(x, "x")
    dt = _dtype(x, "x")
    _norm_params("weight", weight, x, D)
    _norm_params("bias", bias, x, D)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError(f"weight and bias differ in type: {weight.dtype} and {bias.dtype}")
    p = weight if weight is not None else bias
    ld_r = 0
    if residual is not None:
        if residual.shape != x.shape or residual.dtype != x.dtype:
            raise ValueError(f"residual must be {tuple(x.shape)} of {x.dtype}, got "
                             f"{tuple(residual.shape)} of {residual.dtype}")
        ld_r = _rows(residual, "residual", D, x.get_device())[2]
    s = _stream_here(x, stream)
    if s is None:
        with _on(x, stream):
            return layer_norm(x, weight, bias, eps, residual, stats)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    z = torch.empty_like(y) if residual is not None else None
    mean = rstd = None
    if stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    capi.moe_layer_norm(capi.moe_norm_args(
        n, D, dt, dt if p is None else _DTYPES[p.dtype], eps, x.data_ptr(), _ptr(residual),
        _ptr(weight), _ptr(bias), y.data_ptr(), _ptr(z), _ptr(mean), _ptr(rstd), None, None,
        None, None, None, ld, ld_r, D, D), s)
    return y, (x if z is None else z), mean, rstd


def layer_norm_backward(dy, z, weight, mean, rstd, dz=None, bias=True, stream=None):
    """(dx, dweight, dbias) of layer_norm from the gradient dy of y, for the z, mean and
    rstd that it returned. dz: the gradient of z from elsewhere (the residual stream), added
    to dx, which is the gradient of x and of the residual alike. dweight and dbias have the
    weight's type (z's if weight is None, and no dweight then); dbias is None without bias."""
    n, D, ld_z = _rows(z, "z")
    dt = _dtype(z, "z")
    _norm_params("weight", weight, z, D)
    ld = {"dz": 0}
    for t, what in ((dy, "dy"), (dz, "dz")):
        if t is None and what == "dz":
            continue
        if t.shape != z.shape or t.dtype != z.dtype:
            raise ValueError(f"{what} must be {tuple(z.shape)} of {z.dtype}, got {tuple(t.shape)} of "
                             f"{t.dtype}")
        ld[what] = _rows(t, what, D, z.get_device())[2]
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        if (t.shape != z.shape[:-1] or t.dtype != torch.float32 or not t.is_contiguous() or
                t.device != z.device):
            raise ValueError(f"{what} must be contiguous fp32 of shape {tuple(z.shape[:-1])}, got "
                             f"{tuple(t.shape)} of {t.dtype}")
    wt = z.dtype if weight is None else weight.dtype
    s = _stream_here(z, stream)
    if s is None:
        with _on(z, stream):
            return layer_norm_backward(dy, z, weight, mean, rstd, dz, bias)
    dx = torch.empty(z.shape, dtype=z.dtype, device=z.device)
    dw = None if weight is None else torch.empty(D, dtype=wt, device=z.device)
    db = torch.empty(D, dtype=wt, device=z.device) if bias else None
    size = capi.moe_layer_norm_workspace(n, D)
    work = torch.empty(size, dtype=torch.uint8, device=z.device)
    capi.moe_layer_norm_backward(capi.moe_norm_args(
        n, D, dt, _DTYPES[wt], 0.0, None, None, _ptr(weight), None, None, z.data_ptr(),
        mean.data_ptr(), rstd.data_ptr(), dy.data_ptr(), _ptr(dz), dx.data_ptr(), _ptr(dw),
        _ptr(db), 0, 0, 0, ld_z, ld["dy"], ld["dz"], D), work.data_ptr(), size, s)
    return dx, dw, db


# ------------------------------------------------------------------------------- linear
def _operand(t, what, cols, dtype, dev):
    """Rows of a matrix that the tensor maps read: on 16 bytes."""
    n, c, ld = _rows(t, what, cols, dev)
    if t.dtype != dtype:
        raise ValueError(f"{what} has type {t.dtype}: expected {dtype}")
    if t.data_ptr() % 16 or (n > 1 and ld % 8):
        raise ValueError(f"{what} must have rows that start on 16 bytes (a row stride that is a "
                         f"multiple of 8 elements), got a stride of {ld} and an address of "
                         f"{t.data_ptr() % 16} modulo 16")
    return n, c, ld


def _act(act):
    if act not in _ACTS:
        raise ValueError(f"act {act!r}: expected one of {', '.join(_ACTS)}")
    return _ACTS[act]


def linear(x, weight, bias=None, act="none", residual=None, preact=False, out_dtype=None,
           stream=None):
    """(y, z): z = x weight^T + bias, y = act(z) + residual, with fp32 sums.

    x: [..., K], weight: [N, K], both bf16 or both fp16, rows on 16 bytes; bias: [N] of that
    type or fp32; act: "none", "relu", "gelu", "gelu_tanh" or "silu"; residual: [..., N] of
    x's type. y has out_dtype (x's type or fp32; default x's), z (with preact, for
    linear_backward, else None) x's type; both are contiguous."""
    dt, dev, xt = _dtype(x, "x", _HALF), x.get_device(), x.dtype
    M, K, ld_x = _operand(x, "x", None, xt, dev)
    if weight.dim() != 2:
        raise ValueError(f"weight must be [N, K], got {tuple(weight.shape)}")
    N, _, ld_w = _operand(weight, "weight", K, xt, dev)
    a = _act(act)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype not in (x.dtype, torch.float32):
        raise ValueError(f"out_dtype {out_dtype}: expected {x.dtype} or torch.float32")
    if bias is not None:
        _vector(bias, "bias", N, (xt, torch.float32), dev)
    shape, ld_r = (M, N) if x.dim() == 2 else (*x.shape[:-1], N), 0
    if residual is not None:
        if residual.shape != shape or residual.dtype != x.dtype:
            raise ValueError(f"residual must be {shape} of {x.dtype}, got {tuple(residual.shape)} of "
                             f"{residual.dtype}")
        ld_r = _rows(residual, "residual", N, dev)[2]
    s = _stream_here(x, stream)
    if s is None:
        with _on(x, stream):
            return linear(x, weight, bias, act, residual, preact, out_dtype)
    y = torch.empty(shape, dtype=out_dtype, device=x.device)
    z = torch.empty(shape, dtype=x.dtype, device=x.device) if preact else None
    capi.moe_linear(capi.moe_linear_args(
        M, N, K, dt, _DTYPES[out_dtype], dt if bias is None else _DTYPES[bias.dtype], dt, a,
        x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(), _ptr(z), None,
        None, None, None, ld_x, ld_w, ld_r, N, N), s)
    return y, z


def linear_backward(dy, x, weight, z=None, act="none", bias=None, dw_dtype=None, need_dx=True,
                    need_dw=True, stream=None):
    """(dx, dweight, dbias) of linear from the gradient dy of y (which is the residual's
    gradient too), for its x, weight, act and the z that it returned with preact.

    bias: the type of dbias (x's or torch.float32), or None for no dbias. dweight has
    dw_dtype (x's type or fp32; default x's). The products take dy act'(z) rounded to x's
    type."""
    dt, dev, xt = _dtype(x, "x", _HALF), x.get_device(), x.dtype
    M, K, ld_x = _operand(x, "x", None, xt, dev)
    if weight.dim() != 2:
        raise ValueError(f"weight must be [N, K], got {tuple(weight.shape)}")
    N, _, ld_w = _operand(weight, "weight", K, xt, dev)
    a = _act(act)
    shape = (M, N) if x.dim() == 2 else (*x.shape[:-1], N)
    if (z is None) != (a == capi.MOE_ACT_NONE):
        raise ValueError("z is needed with an activation, and only then")
    ld = {"z": 0}
    for t, what in ((dy, "dy"), (z, "z")):
        if t is None:
            continue
        if t.shape != shape or t.dtype != x.dtype:
            raise ValueError(f"{what} must be {shape} of {x.dtype}, got {tuple(t.shape)} of {t.dtype}")
        ld[what] = _rows(t, what, N, dev)[2]
    dw_dtype = x.dtype if dw_dtype is None else dw_dtype
    for t, what in ((dw_dtype, "dw_dtype"), (bias, "bias")):
        if t is not None and t not in (x.dtype, torch.float32):
            raise ValueError(f"{what} {t}: expected {x.dtype} or torch.float32")
    s = _stream_here(x, stream)
    if s is None:
        with _on(x, stream):
            return linear_backward(dy, x, weight, z, act, bias, dw_dtype, need_dx, need_dw)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_dx else None
    dw = torch.empty(N, K, dtype=dw_dtype, device=x.device) if need_dw else None
    db = torch.empty(N, dtype=bias, device=x.device) if bias is not None else None
    size = capi.moe_linear_workspace(M, N)
    work = torch.empty(size, dtype=torch.uint8, device=x.device)
    capi.moe_linear_backward(capi.moe_linear_args(
        M, N, K, dt, dt, dt if bias is None else _DTYPES[bias], _DTYPES[dw_dtype], a, x.data_ptr(),
        weight.data_ptr(), None, None, None, _ptr(z), dy.data_ptr(), _ptr(dx), _ptr(dw), _ptr(db),
        ld_x, ld_w, 0, 0, ld["z"], ld["dy"], K, K), work.data_ptr(), size, s)
    return dx, dw, db


def status(stream=None):
    """(code, detail) of the products' device status: 0, or MOE_DEV_TIMEOUT after a device
    wait ran out. Synchronises the stream; clear_status() clears it."""
    return capi.moe_ops_status((stream or torch.cuda.current_stream()).cuda_stream)


def clear_status(stream=None):
    capi.moe_ops_status_clear((stream or torch.cuda.current_stream()).cuda_stream)
