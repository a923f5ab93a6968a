"""block.MoEBlock: the operators and the routed experts together, as a block runs them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import ops_ref as R  # noqa: E402
from tile_signaled_grouped_gb300 import ops  # noqa: E402
from tile_signaled_grouped_gb300.block import MoEBlock  # noqa: E402
from tile_signaled_grouped_gb300.runtime import ExpertCombine  # noqa: E402
from tile_signaled_grouped_gb300.workloads import get_workload, make_inputs  # noqa: E402

H = 384  # hidden size of the dense expert


def make(bias=True):
    wl = get_workload("tiny")
    inp = make_inputs(wl, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)

    def rnd(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    d = wl.d_model
    layer = ExpertCombine(wl.W, wl.L, wl.topk, wl.T, d, wl.d_ff, wl.tb_M)
    cfg = ops.router_cfg(wl.E, wl.topk, score="sigmoid", groups=4, topk_groups=2, group_top=2,
                         renorm=True, scale=2.5)
    blk = MoEBlock(layer, cfg, 1 + rnd(d, std=0.2), rnd(d, std=0.2) if bias else None,
                   rnd(wl.E, d, std=d ** -0.5), rnd(H, d, std=d ** -0.5),
                   rnd(H, std=0.2, dtype=torch.float32) if bias else None, rnd(d, H, std=H ** -0.5),
                   rnd(d, std=0.2, dtype=torch.float32) if bias else None, inp.w_gate, inp.w_up,
                   inp.w_down, router_bias=rnd(wl.E, std=0.1, dtype=torch.float32))
    x, r = rnd(wl.W * wl.T, d), rnd(wl.W * wl.T, d)
    torch.cuda.synchronize()
    return wl, inp, blk, x, r


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("bias", [True, False])
def test_forward(bias):
    wl, inp, blk, x, r = make(bias)
    y, moe, saved = blk.forward(x, r, save=True)
    torch.cuda.synchronize()
    assert blk.layer.status() == (0, 0) and ops.status() == (0, 0)
    # h, then everything from the stored h (each stage is tested by itself to its roundings).
    s = x.double() + r.double()
    h = torch.nn.functional.layer_norm(s, s.shape[1:], blk.norm_w.double(),
                                       None if blk.norm_b is None else blk.norm_b.double(), blk.eps)
    assert rel(saved["h"], h) < 2.0 ** -8
    h = saved["h"].double()
    ids, w = R.route((h @ blk.w_router.double().t()).cpu().numpy(), wl.topk, "sigmoid",
                     blk.router_bias.double().cpu().numpy(), 4, 2, 2, True, 2.5)
    got = saved["ids"].cpu().numpy()
    # A score differs from its float64 value by its fp32 sums; two tokens of 256 may lie that close.
    assert (got == ids).all(axis=1).sum() >= len(got) - 2
    ids = saved["ids"].long()
    w = torch.tensor(R.weights((h @ blk.w_router.double().t()).cpu().numpy(), got, "sigmoid", True, 2.5),
                     device="cuda")
    wg, wu, wd = (torch.cat(list(t)).double() for t in (inp.w_gate, inp.w_up, inp.w_down))
    want = torch.zeros_like(h)
    for j in range(wl.topk):
        e = ids[:, j]
        hid = R.act(torch.einsum("nd,nfd->nf", h, wg[e]), "silu") * torch.einsum("nd,nfd->nf", h, wu[e])
        want += w[:, j:j + 1] * torch.einsum("nf,ndf->nd", hid, wd[e])
    assert rel(moe, want) < 5e-3  # h and y of an expert are stored in bf16, and so is the sum
    b1 = 0 if blk.b1 is None else blk.b1.double()
    b2 = 0 if blk.b2 is None else blk.b2.double()
    a = R.act(h @ blk.w1.double().t() + b1, "silu")
    assert rel(saved["a"], a) < 2.0 ** -8
    assert rel(y, saved["a"].double() @ blk.w2.double().t() + b2 + s.bfloat16().double()) < 2.0 ** -8
    y2, moe2, none = blk.forward(x, r)
    assert none is None and torch.equal(y, y2) and torch.equal(moe, moe2)
    with pytest.raises(ValueError, match="x must be"):
        blk.forward(x[:10])


def test_backward_is_the_gradient():
    wl, inp, blk, x, r = make()
    dy = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(2),
                     device="cuda").bfloat16()
    y, moe, saved = blk.forward(x, r, save=True)
    d_w = torch.randn(x.shape[0], wl.topk, device="cuda")
    g = blk.backward(dy, saved, d_w=d_w)
    p = {k: getattr(blk, k).double().requires_grad_() for k in ("norm_w", "norm_b", "w_router", "w1", "b1",
                                                                "w2", "b2")}
    s = (x.double() + r.double()).requires_grad_()
    F = torch.nn.functional
    h = F.layer_norm(s, s.shape[1:], p["norm_w"], p["norm_b"], blk.eps)
    out = F.linear(F.silu(F.linear(h, p["w1"], p["b1"])), p["w2"], p["b2"]) + s
    t = F.logsigmoid(F.linear(h, p["w_router"])).gather(1, saved["ids"].long())
    loss = (out * dy.double()).sum() + (2.5 * torch.softmax(t, 1) * d_w.double()).sum()
    names = ["norm_w", "norm_b", "w_router", "w1", "b1", "w2", "b2"]
    want = torch.autograd.grad(loss, [s] + [p[k] for k in names])
    # Seven values on the way are stored in bf16 (s, h, z, a, da, dz, dh), half a step each.
    for k, v in zip(["x"] + names, want):
        assert rel(g[k], v) < 7 * 2.0 ** -9, k


def test_captured_forward_follows_its_input():
    wl, inp, blk, x, r = make()
    blk.forward(x, r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, moe, _ = blk.forward(x, r)
    x.copy_(torch.randn(x.shape, device="cuda").bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    got = y.clone(), moe.clone()
    want = blk.forward(x, r)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("make_empty", [
    lambda n: torch.zeros(n, 16, device="cuda")[:, :0].t(),             # [0, n], columns apart
    lambda n: torch.zeros(1, n, device="cuda").expand(3, n)[None][:0],  # [0, 3, n], one row thrice
    lambda n: torch.zeros(1, n, device="cuda").expand(0, n),
], ids=["transposed", "expanded", "none"])
def test_no_rows_whatever_the_strides(make_empty):
    e = make_empty(8)
    lead = tuple(e.shape[:-1])
    ids, w = ops.route_experts(e, 2)
    assert ids.shape == lead + (2,) and w.shape == lead + (2,)
    assert ops.route_experts_backward(w, e, ids).shape == e.shape
    one = torch.ones(8, device="cuda")
    y, z, mean, rstd = ops.layer_norm(e, one, one, residual=e, stats=True)
    assert y.shape == z.shape == e.shape and mean.shape == lead
    dx, dw, db = ops.layer_norm_backward(e, e, one, mean, rstd, dz=e)
    assert dx.shape == e.shape and not dw.any() and not db.any()
    x, r = e.bfloat16(), make_empty(24).bfloat16()
    y, z = ops.linear(x, torch.ones(24, 8, device="cuda").bfloat16(), act="silu", residual=r, preact=True)
    assert y.shape == z.shape == lead + (24,)
    dx, dw, db = ops.linear_backward(r, x, torch.ones(24, 8, device="cuda").bfloat16(), z=r, act="silu",
                                     bias=torch.float32)
    assert dx.shape == x.shape and not dw.any() and not db.any()


def test_status_of_every_kind_of_stream():
    st = torch.cuda.Stream()
    for stream in (None, st, st.cuda_stream, 0, torch.cuda.default_stream()):
        ops.clear_status(stream)
        assert ops.status(stream) == (0, 0)
