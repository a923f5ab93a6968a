"""block.Experts and MoEBlock with it: the operators on expert rows together, against float64 and the layer,
captured into a graph, on two streams, and the example."""
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import ops_ref as R  # noqa: E402
from tests.test_gpu_ops_block import make, rel  # noqa: E402
from tile_signaled_grouped_gb300 import ops  # noqa: E402
from tile_signaled_grouped_gb300.block import Experts  # noqa: E402


def experts(seed, E, F, D, T, topk, dtype=torch.bfloat16, act="silu", keep="whole", drop=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
    ex = Experts(rnd(E, F, D, std=D ** -0.5), rnd(E, F, D, std=D ** -0.5), rnd(E, D, F, std=F ** -0.5), act=act,
                 keep=keep)
    h = rnd(T, D)
    ids = torch.randn(T, E, generator=g, device="cuda").topk(topk, dim=1).indices.int()
    if drop:
        ids[torch.rand(T, topk, generator=g, device="cuda") < 0.25] = -1
    w = torch.rand(T, topk, generator=g, device="cuda")
    return ex, h, ids, w, rnd(T, D)


def formula(ex, h, ids, w, act):
    """y in float64 as a differentiable function of h, w and the weights."""
    y = torch.zeros_like(h)
    for e in range(ex[0].shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        a = R.act(h[t] @ ex[0][e].t(), act) * (h[t] @ ex[1][e].t())
        y = y.index_add(0, t, w[t, j, None] * (a @ ex[2][e].t()))
    return y


CASES = [(8, 64, 128, 1, 2, torch.bfloat16, "silu", False), (5, 40, 72, 37, 3, torch.float16, "gelu", True),
         (16, 384, 256, 700, 4, torch.bfloat16, "silu", False), (3, 256, 520, 900, 1, torch.bfloat16, "gelu_tanh", True)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward_are_the_formulas(case):
    E, F, D, T, topk, dtype, act, drop = case
    ex, h, ids, w, dy = experts(1, E, F, D, T, topk, dtype, act, drop=drop)
    y, saved = ex.forward(h, ids, w, save=True)
    p = [t.double().requires_grad_() for t in (ex.w_gate, ex.w_up, ex.w_down, h, w)]
    want = formula(p[:3], p[3], ids, p[4], act)
    # Values of 16 bits on the way: gate, up, a, an expert's row and y, half a step each.
    step = 2.0 ** -9 if dtype == torch.bfloat16 else 2.0 ** -12
    assert rel(y, want.detach()) < 5 * step
    assert torch.equal(ex.forward(h, ids, w)[0], y)
    g = ex.backward(dy, saved)
    grads = torch.autograd.grad(want, p, dy.double())
    # And: their gradients dr, da, dgate, dup, dx twice, dh (relative to norms that the sums keep).
    for k, v in zip(("w_gate", "w_up", "w_down", "h", "w"), grads):
        if k == "w":  # dw = <dy, r>, whose terms may cancel: r's errors, relative to |r|, give it |dy| times them
            size = torch.zeros_like(v)
            for j in range(topk):
                t = torch.nonzero(saved["order"].rows[:, j] >= 0)[:, 0]
                r = saved["r"][saved["order"].rows[t, j].long()].double()
                size[t, j] = dy[t].double().norm(dim=1) * r.norm(dim=1)
            assert (g[k].double() - v).norm() < 12 * step * size.norm()
        else:
            assert rel(g[k], v) < 12 * step, k
    assert ops.status() == (0, 0)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward_from_8_bits(case):
    """The same bits as from the restored values, where those are kept whole in fp32's place: dw of the routing
    from the restored rows, and the others within 16-bit roundings of the formula at the restored gate and up."""
    E, F, D, T, topk, dtype, act, drop = case
    ex, h, ids, w, dy = experts(2, E, F, D, T, topk, dtype, act, keep="8 bits", drop=drop)
    y, saved = ex.forward(h, ids, w, save=True)
    y2, whole = Experts(ex.w_gate, ex.w_up, ex.w_down, act=act, keep="whole").forward(h, ids, w, save=True)
    assert torch.equal(y, y2)
    for k in ("gate", "up", "r"):
        alone = ops.checkpoint(whole[k])
        assert torch.equal(saved[k].codes.view(torch.uint8), alone.codes.view(torch.uint8))
        assert torch.equal(saved[k].scales, alone.scales)
    g, order = ex.backward(dy, saved), saved["order"]
    # restored rows have four significant bits: exact in 16 bits unless they leave fp16's range
    back = {k: ops.restore(saved[k], dtype) for k in ("gate", "up", "r")}
    if dtype == torch.bfloat16:
        same = ex.backward(dy, {**whole, **back})
        for k in g:
            assert torch.equal(g[k], same[k]), k
    # 8 bits move a value by 2^-4 of itself at most: the gradients stay near the whole ones.
    near = ex.backward(dy, whole)
    for k in g:
        if k != "w" or T > 1:  # one token's dw may be small against its terms
            assert rel(g[k], near[k].double()) < 2.0 ** -3, k
    assert int(order.offsets[-1]) == int((ids >= 0).sum())


def test_the_block_trains_its_experts():
    wl, inp, blk, x, r = make()
    ex = Experts(*(torch.cat(list(t)) for t in (inp.w_gate, inp.w_up, inp.w_down)), keep="whole")
    y0, moe0, _ = blk.forward(x, r)
    blk.experts = ex
    blk.w_gate, blk.w_up, blk.w_down = ex.ranks(wl.W)
    y1, moe1, _ = blk.forward(x, r)  # the layer, on views of the experts' weights
    assert torch.equal(y0, y1) and torch.equal(moe0, moe1)
    y, moe, saved = blk.forward(x, r, save=True)
    assert torch.equal(y, y0)
    assert rel(moe, moe0.double()) < 4 * 2.0 ** -9  # gate and up are rounded here, not in the layer
    gen = torch.Generator(device="cuda").manual_seed(3)
    dy, d_moe = (torch.randn(x.shape, generator=gen, device="cuda").bfloat16() for _ in range(2))
    g = blk.backward(dy, saved, d_moe=d_moe)
    names = ["norm_w", "norm_b", "w_router", "w1", "b1", "w2", "b2"]
    p = {k: getattr(blk, k).double().requires_grad_() for k in names}
    pe = [t.double().requires_grad_() for t in (ex.w_gate, ex.w_up, ex.w_down)]
    s = (x.double() + r.double()).requires_grad_()
    F = torch.nn.functional
    h = F.layer_norm(s, s.shape[1:], p["norm_w"], p["norm_b"], blk.eps)
    out = F.linear(F.silu(F.linear(h, p["w1"], p["b1"])), p["w2"], p["b2"]) + s
    t = F.logsigmoid(F.linear(h, p["w_router"])).gather(1, saved["ids"].long())
    m = formula(pe, h, saved["ids"], 2.5 * torch.softmax(t, 1), "silu")
    loss = (out * dy.double()).sum() + (m * d_moe.double()).sum()
    want = torch.autograd.grad(loss, [s] + [p[k] for k in names] + pe)
    # Values of 16 bits on the longest way: s, h, gate, up, a, the expert's row, and back dr, da, dgate
    # and dup, dx twice, dh, the scores' gradient, dz, the sums of dh: 16 half steps.
    for k, v in zip(["x"] + names + ["w_gate", "w_up", "w_down"], want):
        assert rel(g[k], v) < 16 * 2.0 ** -9, k
    with pytest.raises(ValueError, match="d_moe"):
        blk.backward(dy, {**saved, "routed": None}, d_moe=d_moe)


def step_of(seed, keep, shape):
    ex, h, ids, w, dy = experts(seed, *shape, keep=keep, drop=seed % 2 == 1)

    def step():
        y, saved = ex.forward(h, ids, w, save=True)
        g = ex.backward(dy, saved)
        # and a dense product beside them, its input kept in 8 bits
        lin = ops.linear_backward(y, ops.checkpoint(h), ex.w_down[0] @ ex.w_gate[0])
        return (y, *g.values(), *lin[:2])

    return step, (h, ids, w, dy)


@pytest.mark.parametrize("keep", ["8 bits", "whole"])
def test_a_captured_step_follows_its_inputs(keep):
    step, (h, ids, w, dy) = step_of(4, keep, (12, 136, 264, 500, 3))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        h.copy_(torch.randn(h.shape, generator=g, device="cuda").to(h.dtype))
        dy.copy_(torch.randn(h.shape, generator=g, device="cuda").to(h.dtype))
        w.copy_(torch.rand(w.shape, generator=g, device="cuda"))
        # other experts, some tokens all of one: the graph holds no sizes of theirs
        ids.copy_(torch.randint(-1, 12 if seed else 2, ids.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ops.status() == (0, 0)


@pytest.mark.parametrize("threads", [False, True], ids=["one thread", "two threads"])
def test_two_streams_with_their_own_data(threads):
    shapes = [(40, 264, 512, 1100, 4), (7, 128, 328, 2300, 2)]
    steps = [step_of(5 + i, "8 bits", s)[0] for i, s in enumerate(shapes)]
    want = []
    for s in steps:
        want.append(s())
        torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in steps], [[], []]

    def run(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(8):
                got[i].append(steps[i]())

    if threads:
        ts = [threading.Thread(target=run, args=(i,)) for i in range(2)]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
    else:
        for i in range(2):
            run(i)
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 8
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    assert ops.status() == (0, 0)


def test_a_stream_given_to_every_call():
    """stream= allocates and runs on that stream, a torch stream or a raw handle."""
    ex, h, ids, w, dy = experts(9, 6, 128, 256, 50, 2)
    order = ops.sort_experts(ids, 6)
    x = ops.expert_rows(h, order)
    gate = ops.expert_linear(x, ex.w_gate, order.offsets)
    c = ops.checkpoint(gate)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    calls = [lambda s: ops.sort_experts(ids, 6, stream=s), lambda s: (ops.expert_rows(h, order, stream=s),),
             lambda s: (ops.expert_rows_backward(x, order, stream=s),),
             lambda s: (ops.combine_experts(x, w, order, stream=s),),
             lambda s: ops.combine_experts_backward(dy, x, w, order, stream=s),
             lambda s: (ops.expert_linear(x, ex.w_gate, order.offsets, stream=s),),
             lambda s: ops.expert_linear_backward(gate, x, ex.w_gate, order.offsets, stream=s),
             lambda s: ops.checkpoint(gate, stream=s), lambda s: (ops.restore(c, torch.bfloat16, stream=s),),
             lambda s: ops.gated(gate, gate, stream=s)[:1],
             lambda s: ops.gated_backward(gate, c, c, need_h=True, stream=s)]
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        for s in (st, st.cuda_stream):
            got = call(s)
            st.synchronize()
            bits = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t  # noqa: E731
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))


def test_the_example_runs():
    out = subprocess.run([sys.executable, "examples/moe_block.py"], capture_output=True, text=True, timeout=240)
    assert out.returncode == 0, out.stderr
    assert "w_down" in out.stdout and "experts of 3 tokens" in out.stdout and "nan" not in out.stdout
