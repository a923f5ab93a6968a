"""Routing to experts (ops.route_experts and its backward) against float64.

The ids have to be those of 64-bit arithmetic everywhere: bf16 scores tie, and scores with
a bias are drawn so that many neighbours lie within a rounding of fp32. Weights and
gradients are held to the rounding errors of their formulas."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import ops_ref as R  # noqa: E402
from tile_signaled_grouped_gb300 import capi, ops  # noqa: E402

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ROUND = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}

# n, E, topk, score, bias, groups, topk_groups, group_top, renorm, scale, dtype
CASES = [
    (1, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "fp32"),
    (515, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "bf16"),
    (130, 128, 8, "softmax", False, 1, 1, 1, True, 1.0, "fp32"),
    (67, 8, 2, "softmax", False, 1, 1, 1, False, 1.0, "fp32"),
    (33, 1, 1, "softmax", True, 1, 1, 1, True, 2.0, "fp16"),
    (9, 33, 32, "sigmoid", True, 1, 1, 1, False, 1.0, "fp32"),
    (64, 40, 32, "softmax", True, 1, 1, 1, False, 1.0, "fp32"),
    (70, 32, 32, "sigmoid", True, 32, 32, 1, True, 1.0, "fp32"),
    (70, 60, 6, "softmax", True, 5, 3, 2, True, 16.0, "fp16"),
    (41, 96, 7, "softmax", False, 3, 2, 2, False, 1.0, "bf16"),
    (41, 96, 7, "sigmoid", False, 32, 9, 2, False, 1.0, "fp32"),
    (41, 24, 3, "sigmoid", False, 24, 5, 2, True, 1.0, "bf16"),
    (50, 300, 10, "sigmoid", True, 10, 4, 1, True, 1.0, "fp32"),
    (50, 1024, 32, "softmax", True, 32, 8, 2, True, 1.0, "fp32"),
    (50, 1000, 16, "sigmoid", False, 1, 1, 1, True, 1.0, "bf16"),
]


def draw(n, E, dtype, bias, seed, pad=0, mask=0.0):
    g = torch.Generator().manual_seed(seed)
    wide = torch.zeros(n, E + pad)
    wide[:, :E] = torch.randn(n, E, generator=g) * 1.5
    if mask:
        wide[:, :E].masked_fill_(torch.rand(n, E, generator=g) < mask, -float("inf"))
        wide[::7, :E] = -float("inf")
    wide = wide.to(DT[dtype]).cuda()
    b = (torch.randn(E, generator=g) * 0.1).cuda() if bias else None
    return wide[:, :E], b


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def check(l, b, topk, score, groups, tg, gt, renorm, scale, seed=0, dtype="fp32"):
    ids, w = ops.route_experts(l, topk, score=score, bias=b, groups=groups, topk_groups=tg,
                               group_top=gt, renorm=renorm, scale=scale)
    l64, b64 = np64(l), np64(b)
    want, ww = R.route(l64, topk, score, b64, groups, tg, gt, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want)
    tol = R.weight_tolerance(l64, topk)
    assert (np.abs(np64(w) - ww) <= tol * np.abs(ww) + 2e-38).all()

    dw = torch.randn(l.shape[0], topk, generator=torch.Generator().manual_seed(seed + 9)).cuda()
    d = ops.route_experts_backward(dw, l, ids, score=score, renorm=renorm, scale=scale)
    assert d.shape == l.shape and d.dtype == l.dtype
    wd = R.route_backward(np64(dw), l64, want, score, renorm, scale)
    # Each term of r (g - sum g r) carries the weight's error twice; the sum of k terms
    # adds k roundings; then the rounding to the gradient's type.
    g, r = scale * np64(dw), R.weights(l64, want, score, renorm, 1.0)
    p = R.scores(l64, score) if score == "softmax" and not renorm else None
    mag = np.abs(g) + (np.abs(g) * r).sum(1, keepdims=True)
    bound = np.zeros_like(l64)
    if p is not None:
        full = np.zeros_like(l64)
        np.put_along_axis(full, want.astype(np.int64), np.abs(g), axis=1)
        bound = p * (full + (np.abs(g) * r).sum(1, keepdims=True))
    else:
        np.put_along_axis(bound, want.astype(np.int64), r * mag, axis=1)
    bound = bound * (2 * tol + (topk + 8) * R.U32) + ROUND[dtype] * np.abs(wd) + 1e-37
    if dtype == "fp16":
        bound += 2.0 ** -25  # half a step of its subnormal numbers
    assert (np.abs(np64(d) - wd) <= bound).all()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_route(case):
    n, E, topk, score, bias, groups, tg, gt, renorm, scale, dtype = case
    l, b = draw(n, E, dtype, bias, 1)
    check(l, b, topk, score, groups, tg, gt, renorm, scale, 1, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_rows_and_strides(dtype, score, renorm):
    """Masked experts, rows with none left, and rows inside wider ones, at an offset."""
    l, _ = draw(50, 120, dtype, False, 2, pad=3, mask=0.7)
    check(l, None, 6, score, 1, 1, 1, renorm, 1.0, 2, dtype)
    l, _ = draw(50, 121, dtype, False, 3, pad=0, mask=0.3)
    check(l[:, 1:], None, 6, score, 4, 2, 2, renorm, 2.5, 3, dtype)


def test_scores_within_a_rounding_are_decided_as_in_64_bits():
    """Biases that nearly cancel the scores' differences: hundreds of neighbours closer than
    fp32 tells apart, among experts and among groups."""
    n, E = 512, 64
    g = torch.Generator().manual_seed(4)
    base = torch.randn(E, generator=g)
    l = base.expand(n, E) + torch.randn(n, E, generator=g) * 1e-6
    for score in ("sigmoid", "softmax"):
        s = R.scores(base[None].double().numpy(), score)[0]
        b = torch.tensor(0.75 - s, dtype=torch.float32)
        for groups, tg, gt in ((1, 1, 1), (8, 3, 2)):
            check(l.cuda(), b.cuda(), 8, score, groups, tg, gt, True, 1.0)
    # Equal scores and biases: the lower id, without a bias and with one.
    l = torch.zeros(9, E).cuda()
    check(l, None, 8, "softmax", 8, 2, 2, True, 1.0)
    check(l, torch.zeros(E).cuda(), 32, "sigmoid", 1, 1, 1, True, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("topk", [1, 4, 31, 32])
def test_equal_scores_in_front_of_one_that_only_64_bits_tell_apart(dtype, topk):
    """Scores that are all 1 in fp32: experts of equal logits come first in the order of fp32
    and ids, at the border too, and the larger logits behind them have to be found."""
    n, E = 64, 96
    g = torch.Generator().manual_seed(14)
    l = 20.0 + torch.randint(0, 3, (n, E), generator=g).float() * 4
    l[: n // 2, : E // 2] = 20.0
    l[0] = 20.0
    l = l.to(DT[dtype]).cuda()
    b = torch.zeros(E)
    check(l, b.cuda(), topk, "sigmoid", 1, 1, 1, True, 1.0)
    check(l, b.cuda(), topk, "sigmoid", 3, 2, 2, False, 1.0)
    b[::7] = 2.0
    check(l, b.cuda(), topk, "sigmoid", 1, 1, 1, False, 1.0)


def test_biases_that_mask_and_large_ones():
    l, _ = draw(40, 48, "fp32", False, 5)
    b = torch.zeros(48)
    b[5:30] = -float("inf")
    check(l, b.cuda(), 23, "sigmoid", 1, 1, 1, True, 1.0)
    check(l, b.cuda(), 8, "softmax", 4, 3, 2, False, 1.0)
    b = torch.randn(48, generator=torch.Generator().manual_seed(6)) * 1e6
    check(l, b.cuda(), 8, "sigmoid", 4, 2, 2, True, 1.0)


def test_scores_out_of_the_range_of_exp():
    l, _ = draw(20, 16, "fp32", False, 7)
    check(l * 20, None, 4, "softmax", 1, 1, 1, True, 1.0)
    low = (l - 95.0).contiguous()
    ids, w = ops.route_experts(low, 4, score="sigmoid", renorm=True)
    want, ww = R.route(np64(low), 4, "sigmoid", renorm=True)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert (np.abs(np64(w) - ww) <= R.weight_tolerance(np64(low), 4) * ww).all()


def test_nan_scores_come_last_and_show_in_the_weights():
    l, b = draw(16, 64, "fp32", True, 8)
    l = l.clone()
    l[3, ::2] = float("nan")
    l[5] = float("nan")
    for bias in (None, b):
        for groups in (1, 4):
            ids, w = ops.route_experts(l, 4, score="sigmoid", bias=bias, groups=groups,
                                       topk_groups=max(1, groups // 2), group_top=2)
            i = ids.cpu().numpy()
            assert ((i >= 0) & (i < 64)).all() and all(len(set(r)) == 4 for r in i.tolist())
            assert (i[3] % 2 == 1).all() and torch.isfinite(w[3]).all()
            assert torch.isnan(w[5]).all()
            assert torch.isfinite(w[[0, 1, 2, 4, 6]]).all()


def test_other_stream_and_graph():
    l, b = draw(300, 64, "fp32", True, 9)
    ids, w = ops.route_experts(l, 4, score="sigmoid", bias=b, renorm=True)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    ids2, w2 = ops.route_experts(l, 4, score="sigmoid", bias=b, renorm=True, stream=st)
    st.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    ids3, w3 = ops.route_experts(l, 4, score="sigmoid", bias=b, renorm=True, stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(w, w3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gi, gw = ops.route_experts(l, 4, score="sigmoid", bias=b, renorm=True)
    l2, _ = draw(300, 64, "fp32", False, 10)
    l.copy_(l2)
    graph.replay()
    wi, ww = ops.route_experts(l2, 4, score="sigmoid", bias=b, renorm=True)
    assert torch.equal(gi, wi) and torch.equal(gw, ww)


def test_empty_and_more_dimensions():
    ids, w = ops.route_experts(torch.zeros(0, 16, device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    l, _ = draw(24, 16, "fp32", False, 11)
    ids, w = ops.route_experts(l.view(2, 12, 16), 3)
    i2, w2 = ops.route_experts(l, 3)
    assert torch.equal(ids.view(24, 3), i2) and torch.equal(w.view(24, 3), w2)
    d = ops.route_experts_backward(torch.ones_like(w), l.view(2, 12, 16), ids)
    assert d.shape == (2, 12, 16)


def test_ids_out_of_range_have_no_gradient():
    l, _ = draw(8, 16, "fp32", False, 12)
    ids, _ = ops.route_experts(l, 2, score="sigmoid")
    bad = ids.clone()
    bad[2, 1], bad[3, 0] = 99, -5
    dw = torch.ones(8, 2, device="cuda")
    good = ops.route_experts_backward(dw, l, ids, score="sigmoid")
    got = ops.route_experts_backward(dw, l, bad, score="sigmoid")
    good[2, ids[2, 1].long()] = 0
    good[3, ids[3, 0].long()] = 0
    assert torch.equal(got, good)


def test_layer_routes_by_the_rule():
    """ExpertCombine.route_experts fills the layer's ids and weights, and forgets the
    routing of an earlier gate."""
    from tile_signaled_grouped_gb300.runtime import ExpertCombine
    from tile_signaled_grouped_gb300.workloads import get_workload, make_inputs, router_weights

    wl = get_workload("tiny")
    inp = make_inputs(wl, device="cuda")
    torch.cuda.synchronize()
    layer = ExpertCombine(wl.W, wl.L, wl.topk, wl.T, wl.d_model, wl.d_ff, wl.tb_M)
    cfg = ops.router_cfg(wl.E, wl.topk, score="sigmoid", groups=4, topk_groups=2, group_top=2,
                         renorm=True, scale=2.5)
    layer.gate(inp.x, router_weights(wl, device="cuda"))
    ids, w = layer.route_experts(inp.logits, cfg)
    with pytest.raises(capi.MoeError, match="MOE_ERR_ARG"):
        layer.plan_build(inp.x, from_gate=True)
    want, ww = R.route(inp.logits.view(-1, wl.E).double().cpu().numpy(), wl.topk, "sigmoid", None, 4, 2,
                       2, True, 2.5)
    torch.cuda.synchronize()
    assert np.array_equal(ids.view(-1, wl.topk).cpu().numpy(), want)
    assert np.allclose(w.view(-1, wl.topk).cpu().numpy(), ww, rtol=1e-5)
    with pytest.raises(ValueError, match="logits"):
        layer.route_experts(inp.logits[:1], cfg)
    with pytest.raises(capi.MoeError, match="MOE_ERR_ARG"):
        layer.route_experts(inp.logits, ops.router_cfg(wl.E, wl.topk + 1))
    layer.close()
