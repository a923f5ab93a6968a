"""The operators on expert rows (order, rows, combine, products) against float64, within the roundings of
their types and of fp32 sums."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import experts_ref as X  # noqa: E402
from tests import ops_ref as R  # noqa: E402
from tests.test_gpu_ops_linear import DT, close  # noqa: E402
from tile_signaled_grouped_gb300 import ops  # noqa: E402


def gen(*parts):
    return torch.Generator(device="cuda").manual_seed(sum(p * 31 ** i for i, p in enumerate(parts)) % 2 ** 31)


def draw_ids(g, T, E, topk, drop):
    ids = (torch.randn(T, E, generator=g, device="cuda") + 0.7 * torch.randn(E, generator=g, device="cuda")
           ).topk(topk, dim=1).indices.int()
    if drop:
        ids[torch.rand(T, topk, generator=g, device="cuda") < 0.2] = -1
        ids[torch.rand(T, generator=g, device="cuda") < 0.1] = E
    return ids


def matrix(g, n, c, dtype, pad=0, std=1.0):
    """Random [n, c], the first columns of rows that are `pad` elements wider."""
    return (torch.randn(n, c + pad, generator=g, device="cuda") * std).to(DT[dtype])[:, :c]


# -------------------------------------------------------------------------------- order
@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (1, 256, 8), (3, 1024, 32), (37, 11, 3), (512, 8, 2), (513, 8, 8),
                                      (1001, 120, 6), (4097, 1024, 1), (12345, 64, 7), (70001, 257, 10)])
@pytest.mark.parametrize("drop", [False, True])
def test_order(T, E, topk, drop):
    ids = draw_ids(gen(T, E, topk), T, E, topk, drop)
    got = ops.sort_experts(ids, E)
    for a, b in zip(got, X.order(ids, E)):
        assert a.dtype == torch.int32 and torch.equal(a.cpu(), b)


def test_order_of_any_ids():
    """One expert for all, the same expert twice, numbers that are no expert."""
    for ids in ([[0, 0], [0, 0], [0, 0]], [[5, 5], [1, 5], [5, 1]], [[-1, -1]], [[7, -2 ** 31], [2 ** 31 - 1, 3]]):
        t = torch.tensor(ids, dtype=torch.int32, device="cuda")
        for a, b in zip(ops.sort_experts(t, 7), X.order(t, 7)):
            assert torch.equal(a.cpu(), b)
    big = torch.full((9000, 4), 3, dtype=torch.int32, device="cuda")
    big[::2] = 2
    for a, b in zip(ops.sort_experts(big, 4), X.order(big, 4)):
        assert torch.equal(a.cpu(), b)


def test_nothing_to_sort():
    got = ops.sort_experts(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 5)
    assert got.slots.numel() == 0 and got.rows.shape == (0, 4) and got.offsets.tolist() == [0] * 6
    x = torch.empty(0, 16, device="cuda")
    assert ops.expert_rows(x, got).shape == (0, 16)
    r = torch.empty(0, 16, device="cuda")
    w = torch.empty(0, 4, device="cuda")
    assert ops.combine_experts(r, w, got).shape == (0, 16)
    dr, dw = ops.combine_experts_backward(x, r, w, got)
    assert dr.shape == (0, 16) and dw.shape == (0, 4)


# --------------------------------------------------------------------------------- rows
# T, E, topk, D, dtype, pad, drop
ROWS = [
    (1, 256, 8, 7168, "bf16", 0, False), (1, 4, 1, 1, "fp16", 0, False), (2, 9, 9, 3, "fp32", 1, False),
    (37, 11, 3, 70, "fp16", 3, True), (64, 8, 2, 128, "bf16", 0, False), (129, 40, 32, 40, "bf16", 8, True),
    (200, 16, 5, 1000, "fp32", 0, True), (1001, 120, 6, 1531, "fp16", 5, True), (333, 7, 2, 2056, "fp32", 4, False),
    (777, 128, 8, 4096, "bf16", 0, True), (64, 16, 9, 520, "bf16", 0, True),
    # few rows a token, by several vectors of each
    (900, 5, 1, 2056, "bf16", 0, True), (3000, 6, 2, 264, "fp16", 0, True), (500, 7, 3, 1032, "fp32", 0, False),
    (600, 9, 4, 1001, "fp16", 0, True), (700, 8, 1, 4765, "bf16", 0, False), (300, 30, 4, 1537, "fp32", 2, True),
]


@pytest.mark.parametrize("case", ROWS, ids=str)
def test_rows_and_back(case):
    T, E, topk, D, dtype, pad, drop = case
    g = gen(T, E, D)
    ids = draw_ids(g, T, E, topk, drop)
    order = ops.sort_experts(ids, E)
    n, x = T * topk, matrix(g, T, D, dtype, pad)
    r = ops.expert_rows(x, order)
    assert torch.equal(r, X.expert_rows(x, order.rows, n))

    total = int(order.offsets[-1])
    rr = matrix(g, n, D, dtype, pad)
    rr[total:] = float("nan")  # rows that no slot has: nothing may come of them
    w = torch.rand(T, topk, generator=g, device="cuda")
    want, tol = X.combine(rr, w, order.rows)
    y = ops.combine_experts(rr, w, order)
    assert y.dtype == x.dtype and y.shape == x.shape
    close(y, want, tol)
    want, tol = X.combine(rr, None, order.rows)
    close(ops.expert_rows_backward(rr, order), want, tol)

    dy = matrix(g, T, D, dtype, pad)
    want_r, want_w, tol = X.combine_backward(dy, rr, w, order.rows, n)
    dr, dw = ops.combine_experts_backward(dy, rr, w, order)
    close(dr, want_r, R.U32 * want_r.abs())
    close(dw, want_w, tol)
    assert (dw[order.rows < 0] == 0).all() and (dr[total:] == 0).all()

    kept = ops.checkpoint(rr)
    want_r, want_w, tol = X.combine_backward(dy, ops.restore(kept, torch.float32), w, order.rows, n)
    dr8, dw8 = ops.combine_experts_backward(dy, kept, w, order)
    assert torch.equal(dr8, dr)
    close(dw8, want_w, tol)
    assert ops.status() == (0, 0)


def test_more_dimensions_and_gradients_of_the_same_thing():
    """[2, 3, ...] batches; <combine(r), dy> moves by <dr, d> and <dw, d> when r and w move by d."""
    g = gen(5)
    ids = draw_ids(g, 6, 5, 3, True).view(2, 3, 3)
    order = ops.sort_experts(ids, 5)
    x = matrix(g, 6, 24, "fp32").view(2, 3, 24)
    r = ops.expert_rows(x, order)
    w = torch.rand(2, 3, 3, generator=g, device="cuda")
    dy = matrix(g, 6, 24, "fp32").view(2, 3, 24)
    dr, dw = ops.combine_experts_backward(dy, r, w, order)
    y = ops.combine_experts(r, w, order)
    assert y.shape == (2, 3, 24) and dw.shape == (2, 3, 3)
    used = (order.rows >= 0).double()
    # The sum is linear in r and in w: <y, dy> = <dr, r> = <dw, w>.
    dot = (y.double() * dy.double()).sum()
    size = (y.double().abs() * dy.double().abs()).sum() + (w * dw * used).abs().sum()
    assert abs(dot - (dr.double() * r.double()).sum()) <= 300 * R.U32 * size
    assert abs(dot - (dw.double() * w.double() * used).sum()) <= 300 * R.U32 * size
    # and expert_rows' gradient is its transpose
    dx = ops.expert_rows_backward(dr, order)
    a, b = (dr.double() * r.double()).sum(), (dx.double() * x.double()).sum()
    assert abs(a - b) <= 300 * R.U32 * ((dr.double() * r.double()).abs().sum())


# ----------------------------------------------------------------------------- products
# rows of every expert, rows behind the last, N, K, dtype, pad
PRODUCTS = [
    ([1], 0, 8, 8, "bf16", 0),
    ([0, 1, 0], 0, 256, 64, "fp16", 0),
    ([3, 0, 5], 4, 264, 72, "bf16", 8),
    ([1] * 8 + [0] * 50, 0, 2048, 1536, "bf16", 0),
    ([32, 33, 31, 64, 65], 3, 128, 128, "fp16", 0),
    ([255, 256, 257, 1], 0, 520, 200, "bf16", 16),
    ([0, 700, 0, 12, 513, 0], 70, 1000, 264, "fp16", 0),
    ([3000], 0, 136, 1000, "bf16", 0),
    ([17, 2, 90] * 40, 5, 72, 328, "fp16", 8),
    ([5] * 1024, 1, 16, 24, "bf16", 0),
    ([2500, 3, 100], 300, 304, 520, "bf16", 0),
    # sums shared out over pairs, forward and (N large) in dx
    ([1, 0, 1], 0, 256, 7168, "bf16", 0),
    ([40, 0, 300], 9, 264, 2056, "fp16", 8),
    ([3, 2], 1, 8192, 128, "bf16", 0),
    ([700], 0, 4104, 136, "fp16", 0),
    # dW in fp32 by parts of the rows, the last whole or of one row
    ([1536, 0, 769, 768, 2048], 3, 264, 136, "bf16", 0),
]


def experts_case(case, whole=False):
    counts, behind, N, K, dtype, pad = case
    g = gen(len(counts), sum(counts), N, K)
    n, E = sum(counts) + behind, len(counts)
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    if whole:
        m = lambda r, c, std=1: torch.randint(-4, 5, (r, c), generator=g, device="cuda").to(DT[dtype])  # noqa: E731
        return offsets, n, m(n, K), m(E * N, K).view(E, N, K), m(n, N), m(n, K)
    weight = matrix(g, E * N, K, dtype, pad, K ** -0.5)
    return (offsets, n, matrix(g, n, K, dtype, pad), weight.unflatten(0, (E, N)), matrix(g, n, N, dtype, pad),
            matrix(g, n, K, dtype, pad))


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: f"{len(c[0])}x{sum(c[0])}+{c[1]} {c[2:]}")
def test_products(case):
    offsets, n, x, weight, dy, add = experts_case(case)
    E, N, K = weight.shape
    total = int(offsets[-1])
    x[total:] = float("nan")  # rows of no expert
    y = ops.expert_linear(x, weight, offsets)
    assert y.shape == (n, N) and y.dtype == x.dtype
    want, size = X.products(x, weight.transpose(1, 2), offsets)
    close(y, want, 2 * (K + 24) * R.U32 * size)
    dy[total:] = float("nan")
    want, size = X.products(dy, weight, offsets)
    dx, dw = ops.expert_linear_backward(dy, x, weight, offsets)
    close(dx, want, 2 * (N + 24) * R.U32 * size)
    want_w, size_w = X.weights_grad(dy, x, offsets)
    tol = 2 * (max(case[0]) + 24) * R.U32 * size_w
    assert dw.dtype == x.dtype
    close(dw, want_w, tol)
    dx2, dw2 = ops.expert_linear_backward(dy, x, weight, offsets, add=add, dw_dtype=torch.float32)
    assert dw2.dtype == torch.float32
    close(dx2, want + add.double(), 2 * (N + 24) * R.U32 * size + R.U32 * (want + add.double()).abs())
    assert torch.equal(dx2[total:], add[total:])
    close(dw2, want_w, tol)
    only_x, none = ops.expert_linear_backward(dy, x, weight, offsets, need_dw=False)
    assert none is None and torch.equal(only_x, dx)
    none, only_w = ops.expert_linear_backward(dy, x, weight, offsets, need_dx=False)
    assert none is None and torch.equal(only_w, dw)
    assert ops.status() == (0, 0)


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: f"{len(c[0])}x{sum(c[0])}+{c[1]} {c[2:]}")
def test_whole_numbers_are_exact(case):
    """Small integers: every product and sum is exact in fp32; a wrong, missing or doubled element shows."""
    offsets, n, x, weight, dy, add = experts_case(case, whole=True)
    y = ops.expert_linear(x, weight, offsets)
    want, _ = X.products(x, weight.transpose(1, 2), offsets)
    assert torch.equal(y, want.to(x.dtype))
    dx, dw = ops.expert_linear_backward(dy, x, weight, offsets, add=add, dw_dtype=torch.float32)
    want, _ = X.products(dy, weight, offsets)
    total = int(offsets[-1])
    want[:] += add.double()
    assert torch.equal(dx, want.to(x.dtype))
    assert torch.equal(dw.double(), X.weights_grad(dy, x, offsets)[0])
    assert int(offsets[-1]) == total


def test_shared_sums_replayed_beside_other_calls():
    """A sum that pairs share has its parts in a workspace of its call: a captured call, replayed on new values
    between calls on another stream, gives what each alone gives, bit by bit."""
    offsets, n, x, weight, dy, _ = experts_case(([2, 0, 3, 1], 2, 256, 4096, "bf16", 0))
    other = experts_case(([1, 1, 1, 1], 0, 256, 4096, "bf16", 0))
    want_other = ops.expert_linear(other[2], other[3], other[0])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    ops.expert_linear(x, weight, offsets)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = ops.expert_linear(x, weight, offsets)
        dx, _ = ops.expert_linear_backward(x, None, weight.transpose(1, 2).contiguous(), offsets, need_dw=False)
    g = gen(77)
    for counts in ([2, 0, 3, 1], [0, 0, 0, 0], [8, 0, 0, 0], [1, 1, 4, 2]):
        x.copy_(matrix(g, n, 4096, "bf16"))
        offsets.copy_(torch.tensor([0] + counts, device="cuda").cumsum(0).int())
        want = ops.expert_linear(x, weight, offsets)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got_other = [ops.expert_linear(other[2], other[3], other[0]) for _ in range(3)]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and (y[sum(counts):] == 0).all()
        assert torch.equal(dx, want)  # the same product, by the weights the other way round
        assert all(torch.equal(o, want_other) for o in got_other)


def test_bad_rows_stay_in_their_expert():
    """NaN and infinities of one expert's rows reach neither another's rows nor its weights' gradient."""
    case = ([70, 3, 65, 130], 0, 200, 136, "bf16", 0)
    offsets, n, x, weight, dy, _ = experts_case(case)
    y, (dx, dw) = ops.expert_linear(x, weight, offsets), ops.expert_linear_backward(dy, x, weight, offsets)
    for e in range(4):
        a, b = int(offsets[e]), int(offsets[e + 1])
        xb, dyb = x.clone(), dy.clone()
        xb[a:b], dyb[a:b] = float("nan"), float("inf")
        yb, (dxb, dwb) = ops.expert_linear(xb, weight, offsets), ops.expert_linear_backward(dyb, xb, weight, offsets)
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[a:b] = False
        assert torch.equal(yb[keep], y[keep]) and torch.equal(dxb[keep], dx[keep])
        others = [i for i in range(4) if i != e]
        assert torch.equal(dwb[others], dw[others])
        assert not torch.isfinite(dwb[e]).any()


def test_offsets_outside_the_rows_are_left_out():
    """Offsets that do not ascend or leave 0 .. n touch nothing outside the matrices."""
    offsets, n, x, weight, dy, _ = experts_case(([40, 50, 60], 0, 64, 64, "bf16", 0))
    for bad in ([-7, 40, 90, 150], [0, 40, 90, 10 ** 6], [0, 40, 40, 40], [150, 150, 150, 150]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        inside = off.clamp(0, n)
        y = ops.expert_linear(x, weight, off)
        want, size = X.products(x, weight.transpose(1, 2), inside)
        close(y, want, 2 * (64 + 24) * R.U32 * size)
        dx, dw = ops.expert_linear_backward(dy, x, weight, off)
        close(dw, X.weights_grad(dy, x, inside)[0], 2 * (100 + 24) * R.U32 * X.weights_grad(dy, x, inside)[1])
    assert ops.status() == (0, 0)


def test_offsets_that_descend_end_in_order():
    """Experts that claim the same rows: what they write is anyone's, but nothing else is touched and
    the call ends."""
    offsets, n, x, weight, dy, _ = experts_case(([40, 50, 60], 0, 64, 64, "bf16", 0))
    for bad in ([0, 90, 40, 150], [150, 0, 150, 0], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -2 ** 31]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y = ops.expert_linear(x, weight, off)
        dx, dw = ops.expert_linear_backward(dy, x, weight, off)
        torch.cuda.synchronize()
        assert y.shape == (n, 64) and dx.shape == (n, 64) and dw.shape == (3, 64, 64)
    assert ops.status() == (0, 0)


def test_more_than_2_31_elements():
    """Rows whose elements, and weights whose elements, do not fit 32 bits: the last ones are right."""
    T, topk, D, E = 40000, 8, 8192, 16
    ids = draw_ids(gen(T, D), T, E, topk, False)
    order = ops.sort_experts(ids, E)
    x = matrix(gen(T), T, D, "bf16")
    r = ops.expert_rows(x, order)
    assert r.numel() > 2 ** 31
    at = torch.tensor([0, 1, T * topk // 2, T * topk - 2, T * topk - 1], device="cuda")
    assert torch.equal(r[at], x[order.slots[at].long() // topk])
    kept = ops.checkpoint(r)
    some = ops.checkpoint(r[at])
    assert torch.equal(kept.codes[at].view(torch.uint8), some.codes.view(torch.uint8))
    assert torch.equal(kept.scales[at], some.scales)
    h, (g8, _) = ops.gated(r, r, checkpoint=True)
    assert torch.equal(h[at], ops.gated(r[at], r[at])[0])
    assert torch.equal(g8.codes[at].view(torch.uint8), some.codes.view(torch.uint8))
    w = torch.rand(T, topk, device="cuda")
    tok = torch.tensor([0, T // 2, T - 1], device="cuda")
    want, tol = X.combine(r, w[tok], order.rows[tok])
    close(ops.combine_experts(r, w, order)[tok], want, tol)
    dr, dw = ops.combine_experts_backward(x, kept, w, order)
    assert torch.equal(dr[at], (x[order.slots[at].long() // topk].float() * w.view(-1)[order.slots[at].long()][:, None])
                       .bfloat16())
    del r, kept, h, g8, dr
    E, N, K = 40, 8192, 8192  # dW of 2.7e9 elements
    weight = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    weight[-1].normal_(std=K ** -0.5)
    weight[0].normal_(std=K ** -0.5)
    offsets = torch.tensor([0] + [5] * (E - 1) + [12], dtype=torch.int32, device="cuda")
    x, dy = matrix(gen(1), 12, K, "bf16"), matrix(gen(2), 12, N, "bf16")
    y = ops.expert_linear(x, weight, offsets)
    for e, rows in ((0, slice(0, 5)), (E - 1, slice(5, 12))):
        x64, w64 = x[rows].double(), weight[e].double()
        close(y[rows], x64 @ w64.t(), R.product_error(x64, w64.t(), K))
    _, dw = ops.expert_linear_backward(dy, x, weight, offsets, need_dx=False)
    d64, x64 = dy[5:].double(), x[5:].double()
    close(dw[-1], d64.t() @ x64, R.product_error(d64.t(), x64, 7))
    assert not dw[1:-1].any()


def test_no_rows():
    weight = torch.randn(3, 16, 24, device="cuda").bfloat16()
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = torch.empty(0, 24, device="cuda").bfloat16(), torch.empty(0, 16, device="cuda").bfloat16()
    assert ops.expert_linear(x, weight, offsets).shape == (0, 16)
    dx, dw = ops.expert_linear_backward(dy, x, weight, offsets)
    assert dx.shape == (0, 24) and torch.equal(dw, torch.zeros_like(weight))
    # rows, but none of an expert
    x, dy = torch.randn(9, 24, device="cuda").bfloat16(), torch.randn(9, 16, device="cuda").bfloat16()
    assert (ops.expert_linear(x, weight, offsets) == 0).all()
    dx, dw = ops.expert_linear_backward(dy, x, weight, offsets)
    assert (dx == 0).all() and (dw == 0).all()


def test_the_same_bits_every_time():
    offsets, n, x, weight, dy, add = experts_case(([300, 0, 7, 900], 3, 520, 640, "bf16", 0))
    first = (ops.expert_linear(x, weight, offsets), *ops.expert_linear_backward(dy, x, weight, offsets, add=add))
    for _ in range(5):
        again = (ops.expert_linear(x, weight, offsets), *ops.expert_linear_backward(dy, x, weight, offsets, add=add))
        assert all(torch.equal(a, b) for a, b in zip(first, again))
