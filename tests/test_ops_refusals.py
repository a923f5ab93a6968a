"""What the operators around the routed experts refuse, and their float64 test references'
gradients against differences; no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from tests import ops_ref as R
from tile_signaled_grouped_gb300 import build as B

B.build()
from tile_signaled_grouped_gb300 import capi, ops  # noqa: E402

ARG = capi.MOE_ERR_ARG


def router(**kw):
    base = dict(E=16, topk=2, score=0, groups=1, topk_groups=1, group_top=1, renorm=0, scale=1.0)
    base.update(kw)
    return capi.moe_router_cfg(*[base[f] for f, _ in capi.moe_router_cfg._fields_])


@pytest.mark.parametrize("bad", [
    dict(E=0), dict(E=1025), dict(topk=0), dict(topk=17), dict(E=64, topk=33), dict(score=2),
    dict(score=-1), dict(groups=0), dict(groups=3), dict(E=66, groups=33), dict(topk_groups=0),
    dict(topk_groups=2), dict(groups=4, topk_groups=1, topk=5), dict(group_top=0),
    dict(group_top=3), dict(renorm=2), dict(scale=float("nan")), dict(scale=float("inf")),
])
def test_router_refuses_configurations(bad):
    lib = capi.lib()
    c = ctypes.byref(router(**bad))
    assert lib.moe_router(None, c, 64, capi.MOE_FP32, 1, 2048, None, 64, 64, None) == ARG
    assert lib.moe_router_backward(c, 64, 64, 64, capi.MOE_FP32, 1, 2048, 64, 2048, None) == ARG


def test_router_refuses_arguments():
    lib = capi.lib()
    c = ctypes.byref(router())
    ok = dict(plan=None, cfg=c, logits=64, dtype=capi.MOE_FP32, n=1, ld=16, bias=None, ids=64, w=64)
    for bad in (dict(cfg=None), dict(logits=None), dict(logits=66), dict(dtype=3), dict(dtype=-1),
                dict(n=-1), dict(n=1 << 32), dict(ld=15), dict(bias=2), dict(ids=None), dict(ids=65),
                dict(w=None), dict(w=2)):
        a = {**ok, **bad}
        assert lib.moe_router(*a.values(), None) == ARG, bad
    ok = dict(cfg=c, d_w=64, logits=64, ids=64, dtype=capi.MOE_BF16, n=1, ld=16, d=64, ld_d=16)
    for bad in (dict(cfg=None), dict(d_w=None), dict(d_w=66), dict(logits=None), dict(logits=65),
                dict(ids=None), dict(ids=2), dict(dtype=9), dict(n=-1), dict(ld=15), dict(d=None),
                dict(d=65), dict(ld_d=15)):
        a = {**ok, **bad}
        assert lib.moe_router_backward(*a.values(), None) == ARG, bad
    # no rows: nothing to do, whatever the pointers
    assert lib.moe_router(None, c, None, capi.MOE_FP32, 0, 16, None, None, None, None) == 0


def test_route_experts_refuses_tensors():
    l = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.route_experts(l, 2)
    with pytest.raises(ValueError, match="type"):
        ops.route_experts(l.double(), 2)
    with pytest.raises(ValueError, match="rows"):
        ops.route_experts(torch.zeros(16, 4).t(), 2)
    with pytest.raises(ValueError, match="rows"):
        ops.route_experts(torch.zeros(16).expand(4, 16), 2)
    with pytest.raises(ValueError, match="bias"):
        ops.route_experts(l, 2, bias=torch.zeros(8))
    with pytest.raises(ValueError, match="bias"):
        ops.route_experts(l, 2, bias=torch.zeros(16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="score"):
        ops.route_experts(l, 2, score="tanh")
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="ids"):
        ops.route_experts_backward(torch.zeros(4, 2), l, ids.long())
    with pytest.raises(ValueError, match="d_w"):
        ops.route_experts_backward(torch.zeros(4, 3), l, ids)
    with pytest.raises(ValueError, match="ids"):
        ops.route_experts_backward(torch.zeros(3, 2), l, ids[:3])


def differences(f, x, g, h=1e-6):
    """Central differences of sum(f(x) * g) for every element of x."""
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        for sign in (1.0, -1.0):
            y = x.copy()
            y[i] += sign * h
            d[i] += sign * (f(y) * g).sum() / (2 * h)
    return d


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_reference_gradient_is_the_difference(score, renorm):
    rng = np.random.default_rng(3)
    l, dw = rng.normal(size=(3, 12)), rng.normal(size=(3, 4))
    ids, _ = R.route(l, 4, score, renorm=renorm)
    d = R.route_backward(dw, l, ids, score, renorm, 2.5)
    want = differences(lambda v: R.weights(v, ids, score, renorm, 2.5), l, dw)
    assert np.abs(d - want).max() < 1e-8


# ---------------------------------------------------------------------------- layer norm
def norm_args(**kw):
    base = dict(n=1, D=8, dtype=capi.MOE_BF16, wtype=capi.MOE_FP32, eps=1e-5, x=64, w=64, b=64, y=64,
                z=64, mean=64, rstd=64, dy=64, dx=64, dw=64, db=64, ld_x=8, ld_r=8, ld_y=8, ld_z=8,
                ld_dy=8, ld_dz=8, ld_dx=8)
    base.update(kw)
    return capi.moe_norm_args(**base)


NORM_BOTH = [dict(n=-1), dict(n=1 << 32), dict(D=0), dict(D=(1 << 24) + 1), dict(dtype=3),
             dict(dtype=-1), dict(wtype=capi.MOE_FP16), dict(dtype=capi.MOE_FP32, wtype=capi.MOE_BF16),
             dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(w=66), dict(z=65),
             dict(ld_z=7), dict(mean=66), dict(rstd=65)]


@pytest.mark.parametrize("bad", NORM_BOTH + [dict(x=None), dict(x=65), dict(ld_x=7), dict(y=None),
                                             dict(ld_y=7), dict(b=65), dict(r=65), dict(r=64, ld_r=7)])
def test_layer_norm_refuses_arguments(bad):
    assert capi.lib().moe_layer_norm(ctypes.byref(norm_args(**bad)), None) == ARG


@pytest.mark.parametrize("bad", NORM_BOTH + [
    dict(z=None), dict(dy=None), dict(dy=65), dict(ld_dy=7), dict(dx=None), dict(ld_dx=7),
    dict(mean=None), dict(rstd=None), dict(dz=65), dict(dz=64, ld_dz=7), dict(dw=66), dict(db=66)])
def test_layer_norm_backward_refuses_arguments(bad):
    assert capi.lib().moe_layer_norm_backward(ctypes.byref(norm_args(**bad)), 64, 1 << 40, None) == ARG


def test_layer_norm_backward_refuses_workspaces():
    lib = capi.lib()
    a = ctypes.byref(norm_args(n=10))
    size = capi.moe_layer_norm_workspace(10, 8)
    assert size >= 10 * 2 * 8 * 4
    assert lib.moe_layer_norm_backward(a, None, size, None) == ARG
    assert lib.moe_layer_norm_backward(a, 66, size, None) == ARG
    assert lib.moe_layer_norm_backward(a, 64, size - 1, None) == capi.MOE_ERR_WORKSPACE
    assert lib.moe_layer_norm(None, None) == ARG
    assert lib.moe_layer_norm_backward(None, 64, size, None) == ARG
    assert lib.moe_layer_norm(ctypes.byref(norm_args(n=0, x=None, y=None)), None) == 0
    assert capi.moe_layer_norm_workspace(0, 8) == 0


def test_layer_norm_refuses_tensors():
    x, w = torch.zeros(4, 16), torch.ones(16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.layer_norm(x, w)
    for bad, match in ((dict(x=x.double()), "type"), (dict(weight=torch.ones(8)), "weight"),
                       (dict(weight=w.half()), "weight"), (dict(bias=torch.ones(16, 1)), "bias"),
                       (dict(x=x.half(), weight=w, bias=w.half()), "differ"),
                       (dict(residual=x[:2]), "residual"), (dict(residual=x.half()), "residual"),
                       (dict(x=torch.zeros(16, 4).t(), weight=torch.ones(16)), "rows"),
                       (dict(x=torch.tensor(1.0)), "rows")):
        with pytest.raises(ValueError, match=match):
            ops.layer_norm(**{**dict(x=x, weight=w), **bad})
    m = torch.zeros(4)
    ok = dict(dy=x, z=x, weight=w, mean=m, rstd=m)
    for bad, match in ((dict(dy=x.half()), "dy"), (dict(dy=x[:2]), "dy"), (dict(dz=x[:, :8]), "dz"),
                       (dict(mean=m[:2]), "mean"), (dict(rstd=m.double()), "rstd"),
                       (dict(weight=w.half()), "weight"), (dict(z=x.double()), "type")):
        with pytest.raises(ValueError, match=match):
            ops.layer_norm_backward(**{**ok, **bad})


def test_layer_norm_reference_gradient_is_the_difference():
    rng = np.random.default_rng(5)
    x, w, b, dy = (rng.normal(size=s) for s in ((3, 10), (10,), (10,), (3, 10)))
    _, z, mean, rstd = R.layer_norm(x, w, b, 1e-3)
    dx, dw, db = R.layer_norm_backward(dy, z, w, mean, rstd)
    assert np.abs(dx - differences(lambda v: R.layer_norm(v, w, b, 1e-3)[0], x, dy)).max() < 1e-8
    assert np.abs(dw - differences(lambda v: R.layer_norm(x, v, b, 1e-3)[0], w, dy)).max() < 1e-8
    assert np.abs(db - differences(lambda v: R.layer_norm(x, w, v, 1e-3)[0], b, dy)).max() < 1e-8


# -------------------------------------------------------------------------------- linear
def linear_args(**kw):
    base = dict(M=2, N=8, K=8, dtype=capi.MOE_BF16, ytype=capi.MOE_FP32, btype=capi.MOE_FP32,
                dwtype=capi.MOE_FP32, act=capi.MOE_ACT_SILU, x=64, w=64, b=64, y=64, z=64, dy=64,
                dx=64, dw=64, db=64, ld_x=8, ld_w=8, ld_r=8, ld_y=8, ld_z=8, ld_dy=8, ld_dx=8, ld_dw=8)
    base.update(kw)
    return capi.moe_linear_args(**base)


LINEAR_BOTH = [dict(M=-1), dict(M=1 << 31), dict(N=0), dict(N=1 << 31), dict(K=0), dict(K=1 << 31),
               dict(dtype=capi.MOE_FP32), dict(dtype=-1), dict(btype=capi.MOE_FP16), dict(act=-1),
               dict(act=5), dict(x=None), dict(x=72), dict(ld_x=12), dict(ld_x=0), dict(w=None),
               dict(w=72), dict(ld_w=12), dict(ld_w=0), dict(z=65), dict(ld_z=7)]


@pytest.mark.parametrize("bad", LINEAR_BOTH + [
    dict(ytype=capi.MOE_FP16), dict(y=None), dict(y=66), dict(ld_y=7), dict(r=65), dict(r=64, ld_r=7),
    dict(b=66)])
def test_linear_refuses_arguments(bad):
    assert capi.lib().moe_linear(ctypes.byref(linear_args(**bad)), None) == ARG


@pytest.mark.parametrize("bad", LINEAR_BOTH + [
    dict(dwtype=capi.MOE_FP16), dict(z=None), dict(dy=None), dict(dy=65), dict(ld_dy=7), dict(dx=65),
    dict(ld_dx=7), dict(dw=66), dict(ld_dw=7), dict(db=66)])
def test_linear_backward_refuses_arguments(bad):
    assert capi.lib().moe_linear_backward(ctypes.byref(linear_args(**bad)), 256, 1 << 40, None) == ARG


def test_linear_backward_refuses_workspaces():
    lib = capi.lib()
    a = ctypes.byref(linear_args())
    size = capi.moe_linear_workspace(2, 8)
    assert lib.moe_linear_backward(a, None, size, None) == ARG
    assert lib.moe_linear_backward(a, 128, size, None) == ARG
    assert lib.moe_linear_backward(a, 256, size - 1, None) == capi.MOE_ERR_WORKSPACE
    assert lib.moe_linear(None, None) == ARG
    assert lib.moe_linear_backward(None, 256, size, None) == ARG
    assert lib.moe_linear(ctypes.byref(linear_args(M=0, x=None, y=None)), None) == 0
    assert capi.moe_linear_workspace(0, 8) == 0


def test_linear_refuses_tensors():
    h = torch.bfloat16
    x, w = torch.zeros(4, 16, dtype=h), torch.zeros(24, 16, dtype=h)
    with pytest.raises(ValueError, match="CUDA"):
        ops.linear(x, w)
    for bad, match in ((dict(x=x.float()), "type"), (dict(weight=w.half()), "type"),
                       (dict(weight=w[:, :8]), "weight"), (dict(weight=w[0]), "weight"),
                       (dict(x=torch.zeros(4, 18, dtype=h)[:, :16]), "16 bytes"),
                       (dict(x=torch.zeros(4, 32, dtype=h)[:, 4:20]), "16 bytes"),
                       (dict(act="tanh"), "act"), (dict(bias=torch.zeros(16)), "bias"),
                       (dict(bias=torch.zeros(24, dtype=torch.float16)), "bias"),
                       (dict(out_dtype=torch.float16), "out_dtype"),
                       (dict(residual=x), "residual"),
                       (dict(residual=torch.zeros(4, 24)), "residual")):
        with pytest.raises(ValueError, match=match):
            ops.linear(**{**dict(x=x, weight=w), **bad})
    dy = torch.zeros(4, 24, dtype=h)
    for bad, match in ((dict(dy=x), "dy"), (dict(dy=dy.float()), "dy"), (dict(act="silu"), "z"),
                       (dict(z=dy), "z"), (dict(z=dy[:2], act="silu"), "z"),
                       (dict(bias=torch.float16), "bias"), (dict(dw_dtype=torch.float16), "dw_dtype")):
        with pytest.raises(ValueError, match=match):
            ops.linear_backward(**{**dict(dy=dy, x=x, weight=w), **bad})


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_activation_reference_gradient_is_the_difference(kind):
    z = torch.linspace(-7, 7, 141, dtype=torch.float64) + 0.013
    h = 1e-5
    d = (R.act(z + h, kind) - R.act(z - h, kind)) / (2 * h)
    assert (R.act_grad(z, kind) - d).abs().max() < 1e-8


# -------------------------------------------------------------------------------- status
def test_status_takes_streams_and_raw_handles(monkeypatch):
    seen = []
    monkeypatch.setattr(capi, "moe_ops_status", lambda s: seen.append(s) or (0, 0))
    monkeypatch.setattr(capi, "moe_ops_status_clear", seen.append)

    class Stream:
        cuda_stream = 77

    for stream in (Stream(), 78, 0):
        assert ops.status(stream) == (0, 0)
        ops.clear_status(stream)
    assert seen == [77, 77, 78, 78, 0, 0]
