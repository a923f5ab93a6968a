"""The operators on expert rows at the edges of what their documentation allows, into memory that holds NaN
before the call: what a call leaves unwritten shows."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import experts_ref as X  # noqa: E402
from tests import ops_ref as R  # noqa: E402
from tests.test_gpu_ops_experts import draw_ids, experts_case, gen, matrix  # noqa: E402
from tests.test_gpu_ops_linear import DT, close  # noqa: E402
from tile_signaled_grouped_gb300 import capi, ops  # noqa: E402
from tile_signaled_grouped_gb300.block import Experts  # noqa: E402

TYPE = {torch.bfloat16: capi.MOE_BF16, torch.float16: capi.MOE_FP16, torch.float32: capi.MOE_FP32}


def ptr(t):
    return t.data_ptr() if t is not None else None


def c_call(name, cls, workspace=None, **fields):
    """A call of the C ABI on the current stream."""
    a = cls(**{k: ptr(v) if isinstance(v, torch.Tensor) else v for k, v in fields.items()})
    more = () if workspace is None else (ptr(workspace), workspace.numel())
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert getattr(capi.lib(), name)(ctypes.byref(a), *more, stream) == 0


def nan(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def products_into_nan(x, weight, dy, add, offsets):
    """(y, dx, dx with add, dW) by the C ABI, every output full of NaN before its call."""
    E, N, K = weight.shape
    n, t = x.shape[0], x.dtype
    size = capi.lib().moe_expert_linear_workspace
    work = nan(max(size(n, N, K, E), size(n, K, N, E)) // 4 + 4, dtype=torch.float32).view(torch.uint8)
    both = dict(n=n, N=N, K=K, E=E, dtype=TYPE[t], dwtype=capi.MOE_FP32, offsets=offsets, w=weight,
                ld_w=weight.stride(1), stride_w=weight.stride(0))
    y, dx, dx2 = nan(n, N, dtype=t), nan(n, K, dtype=t), nan(n, K, dtype=t)
    dw = nan(E, N, K, dtype=torch.float32)
    c_call("moe_expert_linear", capi.moe_expert_linear_args, work, **both, x=x, ld_x=x.stride(0), y=y, ld_y=N)
    for out, plus in ((dx, None), (dx2, add)):
        c_call("moe_expert_linear_backward", capi.moe_expert_linear_args, work, **both, x=x, ld_x=x.stride(0), dy=dy,
               ld_dy=dy.stride(0), add=plus, ld_add=add.stride(0), dx=out, ld_dx=K, dw=dw, ld_dw=K, stride_dw=N * K)
    return y, dx, dx2, dw


# rows before the first expert's, then as in test_gpu_ops_experts
BEFORE = [
    (1, ([2], 0, 8, 8, "bf16", 0)),
    (40, ([50, 0, 60], 0, 64, 64, "bf16", 0)),
    (300, ([3, 0, 5], 4, 264, 72, "fp16", 8)),
    (2500, ([700, 1], 300, 136, 200, "bf16", 0)),  # more tiles than are walked together
    (17, ([1] * 1024, 3, 16, 24, "bf16", 0)),      # the longest table
    (150, ([0, 0, 0], 0, 64, 64, "bf16", 0)),      # every row
    # sums shared out over pairs, forward and in dx
    (5, ([1, 0, 1], 0, 256, 7168, "bf16", 0)),
    (9, ([3, 2], 1, 8192, 128, "fp16", 0)),
    (6, ([0, 0], 0, 512, 4096, "bf16", 0)),
]


@pytest.mark.parametrize("before,case", BEFORE, ids=lambda v: f"{len(v[0])}x{sum(v[0])}+{v[1]} {v[2:]}"
                         if isinstance(v, tuple) else str(v))
def test_rows_before_the_first_expert_are_zero(before, case):
    """Small integers, so that everything is exact. The offsets of some experts out of more begin above 0: the
    rows before them are zero in y and `add` alone in dx, as those behind the last expert's are."""
    counts, behind, N, K, dtype, pad = case
    _, n, x, weight, dy, add = experts_case((counts, behind + before, N, K, dtype, pad), whole=True)
    offsets = torch.tensor([before] + counts, device="cuda").cumsum(0).int()
    y, dx, dx2, dw = products_into_nan(x, weight, dy, add, offsets)
    want, _ = X.products(x, weight.transpose(1, 2), offsets)
    assert torch.equal(y, want.to(x.dtype))
    want, _ = X.products(dy, weight, offsets)
    assert torch.equal(dx, want.to(x.dtype))
    assert torch.equal(dx2, (want + add.double()).to(x.dtype))
    assert torch.equal(dw.double(), X.weights_grad(dy, x, offsets)[0])
    assert ops.status() == (0, 0)


def test_some_experts_of_an_order():
    """The rows of two halves of the experts, by slices of the offsets and of the weights, add up to those of all."""
    offsets, n, x, weight, dy, add = experts_case(([30, 0, 7, 300, 1, 64], 5, 72, 136, "bf16", 0), whole=True)
    y = ops.expert_linear(x, weight, offsets)
    parts = [ops.expert_linear(x, weight[a:b], offsets[a:b + 1]) for a, b in ((0, 3), (3, 6))]
    assert torch.equal(parts[0] + parts[1], y)
    assert torch.equal(parts[0] != 0, (y != 0) & (torch.arange(n, device="cuda") < 37)[:, None])


def test_offsets_that_leave_no_rows_inside():
    """As test_offsets_outside_the_rows_are_left_out, into NaN, and dx too."""
    _, n, x, weight, dy, add = experts_case(([40, 50, 60], 0, 64, 64, "bf16", 0), whole=True)
    for bad in ([-7, 40, 90, 150], [0, 40, 90, 10 ** 6], [0, 40, 40, 40], [150, 150, 150, 150],
                [7, 7, 10 ** 6, 10 ** 6]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        inside = off.clamp(0, n)
        y, dx, dx2, dw = products_into_nan(x, weight, dy, add, off)
        assert torch.equal(y, X.products(x, weight.transpose(1, 2), inside)[0].to(x.dtype)), bad
        want, _ = X.products(dy, weight, inside)
        assert torch.equal(dx, want.to(x.dtype)) and torch.equal(dx2, (want + add.double()).to(x.dtype)), bad
        assert torch.equal(dw.double(), X.weights_grad(dy, x, inside)[0]), bad
    assert ops.status() == (0, 0)


# e: the type's largest exponent. |x| from 1.9375 2^e on is nearest to 2^(e + 1), which the type does not hold.
TOP = {torch.float16: (15, 65504.0, 63456.0), torch.bfloat16: (127, 3.3895313892515355e38, 1.9296875 * 2.0 ** 127),
       torch.float32: (127, 3.4028234663852886e38, 3.29e38)}


@pytest.mark.parametrize("dtype", TOP, ids=str)
@pytest.mark.parametrize("c", [64, 77, 512])
def test_the_largest_numbers_stay_finite_in_8_bits(dtype, c):
    """A type's largest numbers are kept as 1.875 2^e: 2^-4 of them is what the code loses at most, and the one
    above would come back as an infinity."""
    e, most, below = TOP[dtype]
    x = torch.full((3, c), 2.0 ** (e - 3), device="cuda").to(dtype)
    special = torch.tensor([most, -most, 1.9375 * 2.0 ** e, -1.9375 * 2.0 ** e, below, 1.75 * 2.0 ** e, -0.0, 1.0])
    x[0, :8] = special.to(dtype)
    x[1, c - 8:] = special.to(dtype)
    x[2, 3], x[2, 5] = most, float("inf")  # the others of a block with an infinity
    kept = ops.checkpoint(x)
    back = ops.restore(kept, dtype)
    assert torch.equal(torch.isnan(back), torch.isinf(x)) and not torch.isinf(back).any()
    want = torch.tensor([1.875, -1.875, 1.875, -1.875, 1.875, 1.75], dtype=torch.float64) * 2.0 ** e
    assert torch.equal(back[0, :6].double().cpu(), want) and torch.equal(back[1, c - 8:c - 2].double().cpu(), want)
    assert float(back[2, 3].double()) == 1.875 * 2.0 ** e
    finite = torch.isfinite(x) & (x.abs() > 2.0 ** e / 2 ** 10)
    x64 = x.double()
    assert ((back.double() - x64).abs() <= 2.0 ** -4 * x64.abs())[finite].all()
    if dtype == torch.float32:
        return
    # as gate and up, kept by the launch that multiplies them, and read in place of them
    _, both = ops.gated(x, x, checkpoint=True)
    for k in both:
        assert torch.equal(k.codes.view(torch.uint8), kept.codes.view(torch.uint8))
        assert torch.equal(k.scales, kept.scales)
    small = torch.full_like(x, 2.0 ** -14)
    dg, du, _ = ops.gated_backward(small[:2], *(ops.Checkpoint(k.codes[:2], k.scales[:2]) for k in both), act="relu")
    assert torch.isfinite(dg).all() and torch.isfinite(du).all()


def test_linear_backward_from_the_largest_numbers():
    """dW of an x at the end of fp16's range, from 8 bits: the product of 61440 with the rows' 2^-12."""
    x = torch.full((40, 64), 65504.0, dtype=torch.float16, device="cuda")
    dy = torch.full((40, 16), 2.0 ** -12, dtype=torch.float16, device="cuda")
    w = torch.zeros(16, 64, dtype=torch.float16, device="cuda")
    _, dw, _ = ops.linear_backward(dy, ops.checkpoint(x), w, need_dx=False)
    assert (dw == 40 * 61440 * 2.0 ** -12).all()


# T, E, topk, D, dtype, pad of the rows, pad of dy, drop: rows on 16 bytes, dy's alone elsewhere
DY_ANYWHERE = [(T, E, topk, D, dtype, pad, 1 + 2 * (topk % 3), drop)
               for T, E, topk, D, drop in ((1, 4, 1, 8, False), (300, 5, 1, 2056, True), (257, 6, 2, 264, True),
                                           (100, 9, 4, 1032, False), (77, 30, 8, 4096, True), (64, 16, 11, 520, True))
               for dtype, pad in (("bf16", 0), ("fp16", 8), ("fp32", 4))]


@pytest.mark.parametrize("case", DY_ANYWHERE, ids=str)
def test_combine_gradient_of_a_dy_that_starts_anywhere(case):
    """dy as columns of something wider: the rows go by vectors, dy alone by two of them shifted together. The
    same bits as with a dy of its own, from values and from codes."""
    T, E, topk, D, dtype, pad, pad_dy, drop = case
    g = gen(T, E, D)
    order = ops.sort_experts(draw_ids(g, T, E, topk, drop), E)
    n, total = T * topk, int(order.offsets[-1])
    r, dy = matrix(g, n, D, dtype, pad), matrix(g, T, D, dtype, pad_dy)
    r[total:] = float("nan")
    dy.as_strided((T - 1, pad_dy), (D + pad_dy, 1), dy.storage_offset() + D)[:] = float("nan")  # between its rows
    w = torch.rand(T, topk, generator=g, device="cuda")
    for kept in (r, ops.checkpoint(r)):
        want = ops.combine_experts_backward(dy.clone(memory_format=torch.contiguous_format), kept, w, order)
        for a, b in zip(ops.combine_experts_backward(dy, kept, w, order), want):
            assert torch.equal(a, b)
    want_r, want_w, tol = X.combine_backward(dy, r, w, order.rows, n)
    dr, dw = ops.combine_experts_backward(dy, r, w, order)
    close(dr, want_r, R.U32 * want_r.abs())
    close(dw, want_w, tol)
    # without weights
    ones = torch.ones_like(w)
    assert torch.equal(ops.combine_experts_backward(dy, r, ones, order)[0], ops.expert_rows(dy, order))
    assert ops.status() == (0, 0)


@pytest.mark.parametrize("n,c", [(1, 1), (1, 7), (3, 33), (40, 136), (65, 1531), (7, 4104)])
@pytest.mark.parametrize("at", [(0, 1, 0), (1, 0, 1), (1, 1, 0), (0, 0, 1)], ids=str)
def test_gated_gradients_that_start_in_different_places(n, c, at):
    """By the C ABI, dgate, dup and h in rows of their own, some of them off a word's beginning: the same bits as by
    ops, and nothing beside the rows."""
    g = gen(n, c)
    dt = torch.float16 if c % 2 else torch.bfloat16
    gate, up, dh = (torch.randn(n, c, generator=g, device="cuda").to(dt) for _ in range(3))
    want = ops.gated_backward(dh, gate, up, need_h=True)
    for pads in ((1, 1, 1), (2, 3, 4)):  # rows that all lie alike, and rows that do not
        wide = [nan(n * (c + p) + 2, dtype=dt) for p in pads]
        out = [t[a:a + n * (c + p)].view(n, c + p)[:, :c] for t, a, p in zip(wide, at, pads)]
        c_call("moe_gated_backward", capi.moe_gated_args, n=n, c=c, dtype=TYPE[dt], act=capi.MOE_ACT_SILU, gate=gate,
               up=up, dh=dh, dgate=out[0], dup=out[1], h=out[2], ld_gate=c, ld_up=c, ld_dh=c, ld_dgate=c + pads[0],
               ld_dup=c + pads[1], ld_h=c + pads[2])
        for o, v, t in zip(out, want, wide):
            assert torch.equal(o, v) and int(torch.isnan(t).sum()) == t.numel() - n * c
    assert ops.status() == (0, 0)


def test_a_long_sum_in_fp32_keeps_its_accuracy():
    """dW of 32768 rows of one expert. The rows are taken 768 at a time: 48 steps of the tensor cores, which drop what
    lies below the sum's last bit (2^-23 of it a step at most), and 43 parts, each added with a rounding (2^-24).
    Running sums are no larger than the last, in the norm. In one part it would be 2048 steps, and is 3.8e-5."""
    n, N, K = 32768, 256, 512
    g = gen(n, N, K)
    x, dy = matrix(g, n, K, "bf16"), matrix(g, n, N, "bf16")
    offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    weight = torch.zeros(1, N, K, dtype=torch.bfloat16, device="cuda")
    _, dw = ops.expert_linear_backward(dy, x, weight, offsets, dw_dtype=torch.float32, need_dx=False)
    want = dy.double().t() @ x.double()
    parts = -(-n // 768)
    assert (dw[0].double() - want).norm() <= (48 * 2.0 ** -23 + parts * 2.0 ** -24) * want.norm()


def test_weights_and_rows_that_are_parts_of_others():
    """Gate and up as halves of one matrix of every expert, every other expert of a stack, and x and dy as columns
    of wider rows: the same bits as of copies."""
    counts, E, F, K = [70, 0, 300, 9], 4, 136, 264
    g = gen(E, F, K)
    n = sum(counts)
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    both = matrix(g, 2 * E * 2 * F, K, "bf16", 8, K ** -0.5).unflatten(0, (2 * E, 2 * F))
    wide_x, wide_dy = matrix(g, n, 3 * K, "bf16"), matrix(g, n, 2 * F, "bf16")
    for weight in (both[:E, :F], both[:E, F:], both[::2, :F], both[1::2, F:]):
        x, dy = wide_x[:, K:2 * K], wide_dy[:, F:]
        own = [t.contiguous() for t in (x, dy, weight)]
        assert torch.equal(ops.expert_linear(x, weight, offsets), ops.expert_linear(own[0], own[2], offsets))
        got = ops.expert_linear_backward(dy, x, weight, offsets, add=wide_x[:, :K])
        want = ops.expert_linear_backward(own[1], own[0], own[2], offsets, add=wide_x[:, :K].contiguous())
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ops.status() == (0, 0)


@pytest.mark.parametrize("keep", ["8 bits", "whole"])
def test_experts_of_batches_and_of_nothing(keep):
    """Tokens [2, 3, 5, D] as [30, D]; none at all; none that any expert was chosen for."""
    g = gen(8, 4)
    E, F, D, topk = 6, 40, 72, 3
    weights = [matrix(g, E * a, b, "bf16", 0, b ** -0.5).unflatten(0, (E, a)) for a, b in ((F, D), (F, D), (D, F))]
    ex = Experts(*weights, keep=keep)
    h, dy = matrix(g, 30, D, "bf16"), matrix(g, 30, D, "bf16")
    ids, w = draw_ids(g, 30, E, topk, True), torch.rand(30, topk, generator=g, device="cuda")
    y, saved = ex.forward(h, ids, w, save=True)
    grads = ex.backward(dy, saved)
    shape = (2, 3, 5)
    y4, saved4 = ex.forward(h.view(*shape, D), ids.view(*shape, topk), w.view(*shape, topk), save=True)
    assert y4.shape == (*shape, D) and torch.equal(y4.view(30, D), y)
    for k, v in ex.backward(dy.view(*shape, D), saved4).items():
        assert torch.equal(v.view(grads[k].shape), grads[k]), k

    y, saved = ex.forward(h[:0], ids[:0], w[:0], save=True)
    grads = ex.backward(dy[:0], saved)
    assert y.shape == (0, D) and grads["h"].shape == (0, D) and grads["w"].shape == (0, topk)
    assert not any(grads[k].any() for k in ("w_gate", "w_up", "w_down"))
    y, saved = ex.forward(h, torch.full_like(ids, -1), w, save=True)
    grads = ex.backward(dy, saved)
    assert not y.any() and not any(v.any() for v in grads.values())
    assert ops.status() == (0, 0)


# ------------------------------------------------------------------- outputs inside something wider
class Wide:
    """An output [n, c] from element `at` of a buffer full of one byte, in rows of `ld`; untouched() says that nothing
    beside its rows was written."""

    def __init__(self, n, c, ld, at, dtype, experts=1, stride=0):
        size = torch.empty(0, dtype=dtype).element_size()
        self.bytes = torch.full(((at + (experts - 1) * stride + n * ld + 64) * size,), 0x5A, dtype=torch.uint8,
                                device="cuda")
        self.all = self.bytes.view(dtype)
        self.t = self.all.as_strided((experts, n, c), (stride, ld, 1), at)
        if experts == 1:
            self.t = self.t[0]
        self.n, self.c, self.ld, self.at, self.size, self.experts, self.stride = n, c, ld, at, size, experts, stride

    def untouched(self):
        mask = torch.ones(self.bytes.numel() // self.size, dtype=torch.bool, device="cuda")
        mask.as_strided((self.experts, self.n, self.c), (self.stride, self.ld, 1), self.at)[:] = False
        return bool((self.bytes.view(-1, self.size)[mask] == 0x5A).all())


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,topk,D,pad,at", [(5, 2, 1, 2, 1), (33, 3, 70, 3, 5), (40, 8, 264, 8, 8),
                                             (17, 1, 1531, 5, 3), (50, 4, 520, 1, 0), (29, 2, 33, 31, 7)])
def test_rows_into_wider_rows(T, topk, D, pad, at, dtype):
    """By the C ABI, rows, sums and their gradients inside something wider: the same bits as by ops, and nothing
    beside."""
    g = gen(T, D)
    dt, E, n = DT[dtype], 11, T * topk
    order = ops.sort_experts(draw_ids(g, T, E, topk, True), E)
    x, r, w = matrix(g, T, D, dtype), matrix(g, n, D, dtype), torch.rand(T, topk, generator=g, device="cuda")
    same = dict(T=T, D=D, topk=topk, E=E, dtype=TYPE[dt], rows=order.rows, offsets=order.offsets)
    out = Wide(n, D, D + pad, at, dt)
    c_call("moe_expert_rows", capi.moe_rows_args, **same, x=x, ld_x=D, dr=out.t, ld_dr=out.ld)
    assert torch.equal(out.t, ops.expert_rows(x, order)) and out.untouched()
    for weights in (w, None):
        out = Wide(T, D, D + pad, at, dt)
        c_call("moe_combine_experts", capi.moe_rows_args, **same, w=weights, r=r, ld_r=D, y=out.t, ld_y=out.ld)
        assert torch.equal(bits(out.t), bits(ops.combine_experts(r, weights, order))) and out.untouched()
    kept = ops.checkpoint(r)
    for src, scales in ((r, None), (kept.codes, kept.scales)):
        out, dw = Wide(n, D, D + pad, at, dt), Wide(T, topk, topk, 1, torch.float32)
        c_call("moe_combine_experts_backward", capi.moe_rows_args, **same, w=w, x=x, ld_x=D, r=src, ld_r=D,
               r_scales=scales, ld_scales=-(-D // 32), dr=out.t, ld_dr=out.ld, dw=dw.t)
        want, _ = ops.combine_experts_backward(x, r if scales is None else kept, w, order)
        assert torch.equal(bits(out.t), bits(want)) and out.untouched() and dw.untouched()
        # sums over the columns are shared out by where rows start: within their own errors
        values = r if scales is None else ops.restore(kept, torch.float32)
        close(dw.t, *X.combine_backward(x, values, w, order.rows, n)[1:])
    assert ops.status() == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,c,pad,at", [(1, 1, 0, 1), (3, 31, 2, 3), (5, 64, 32, 8), (9, 136, 8, 16), (40, 1531, 5, 5),
                                        (6, 4096, 1, 0), (65, 128, 5, 0)])
def test_checkpoints_into_wider_rows(n, c, pad, at, dtype):
    """As above, codes and scales in rows of their own, and restored into wider rows from them."""
    dt = DT[dtype]
    x = matrix(gen(n, c), n, c, dtype)
    want, blocks = ops.checkpoint(x), -(-c // 32)
    codes, scales = Wide(n, c, c + pad, at, torch.uint8), Wide(n, blocks, blocks + pad, at, torch.uint8)
    back = Wide(n, c, c + pad, at, dt)
    same = dict(n=n, c=c, dtype=TYPE[dt], codes=codes.t, scales=scales.t, ld_codes=codes.ld, ld_scales=scales.ld)
    c_call("moe_checkpoint", capi.moe_checkpoint_args, **same, x=x, ld_x=c)
    assert torch.equal(codes.t, want.codes.view(torch.uint8)) and torch.equal(scales.t, want.scales)
    c_call("moe_restore", capi.moe_checkpoint_args, **same, x=back.t, ld_x=back.ld)
    assert torch.equal(bits(back.t), bits(ops.restore(want, dt)))
    assert codes.untouched() and scales.untouched() and back.untouched()


@pytest.mark.parametrize("n,c,pad,at", [(1, 1, 0, 1), (3, 33, 2, 3), (9, 136, 8, 16), (40, 1531, 5, 5),
                                        (6, 4104, 1, 0)])
@pytest.mark.parametrize("keep", [False, True])
def test_gated_into_wider_rows(n, c, pad, at, keep):
    """As above; the codes' rows are c apart, from any byte on."""
    g = gen(n, c)
    dt = torch.float16 if c % 2 else torch.bfloat16
    gate, up, dh = (torch.randn(n, c, generator=g, device="cuda").to(dt) for _ in range(3))
    want, kept = ops.gated(gate, up, checkpoint=True)
    blocks = -(-c // 32)
    h = Wide(n, c, c + pad, at, dt)
    parts = [Wide(n, m, m, at, torch.uint8) for m in (c, blocks, c, blocks)] if keep else [None] * 4
    named = dict(zip(("gate_codes", "gate_scales", "up_codes", "up_scales"), (p and p.t for p in parts)))
    both = dict(n=n, c=c, dtype=TYPE[dt], act=capi.MOE_ACT_SILU)
    c_call("moe_gated", capi.moe_gated_args, **both, **named, gate=gate, up=up, ld_gate=c, ld_up=c, h=h.t, ld_h=h.ld)
    assert torch.equal(bits(h.t), bits(want)) and h.untouched()
    if keep:
        for p, v in zip(parts, (*kept[0], *kept[1])):
            assert torch.equal(p.t, v.view(torch.uint8)) and p.untouched()
        gate, up = parts[0].t, parts[2].t
    scales = dict(gate_scales=parts[1].t, up_scales=parts[3].t) if keep else {}
    out = [Wide(n, c, c + pad, at, dt) for _ in range(3)]
    c_call("moe_gated_backward", capi.moe_gated_args, **both, **scales, gate=gate, up=up, ld_gate=c, ld_up=c, dh=dh,
           ld_dh=c, dgate=out[0].t, dup=out[1].t, h=out[2].t, ld_dgate=c + pad, ld_dup=c + pad, ld_h=c + pad)
    src = kept if keep else (gate, up)
    for o, v in zip(out, ops.gated_backward(dh, *src, need_h=True)):
        assert torch.equal(bits(o.t), bits(v)) and o.untouched()
    assert ops.status() == (0, 0)


@pytest.mark.parametrize("case", [([5, 0, 40], 3, 8, 8, "bf16", 0), ([300, 1, 0, 70], 0, 264, 136, "fp16", 0),
                                  ([1000], 9, 200, 1000, "bf16", 0), ([2, 0, 1], 0, 256, 4096, "bf16", 0),
                                  ([1600, 0, 769], 0, 72, 328, "fp16", 0), ([0, 0], 0, 40, 24, "bf16", 0)],
                         ids=lambda c: f"{len(c[0])}x{sum(c[0])}+{c[1]} {c[2:]}")
def test_products_into_wider_rows(case):
    """y and dx in wider rows; dW of every expert in wider rows, experts further apart than they need."""
    offsets, n, x, weight, dy, add = experts_case(case)
    E, N, K = weight.shape
    lib, dt = capi.lib(), x.dtype
    y, dx = Wide(max(n, 1), N, N + 8, 8, dt), Wide(max(n, 1), K, K + 16, 16, dt)
    work = nan(max(lib.moe_expert_linear_workspace(n, N, K, E), lib.moe_expert_linear_workspace(n, K, N, E)) // 4 + 4,
               dtype=torch.float32).view(torch.uint8)
    same = dict(n=n, N=N, K=K, E=E, dtype=TYPE[dt], offsets=offsets, w=weight, ld_w=K, stride_w=N * K)
    if n:
        c_call("moe_expert_linear", capi.moe_expert_linear_args, work, **same, x=x, ld_x=K, y=y.t, ld_y=y.ld)
        assert torch.equal(y.t, ops.expert_linear(x, weight, offsets)) and y.untouched()
    for wt in (dt, torch.float32):
        dw = Wide(N, K, K + 24, 8, wt, E, N * (K + 24) + 40)
        c_call("moe_expert_linear_backward", capi.moe_expert_linear_args, work, **same, dwtype=TYPE[wt], x=x, ld_x=K,
               dy=dy, ld_dy=N, add=add, ld_add=K, dx=dx.t if n else None, ld_dx=dx.ld, dw=dw.t, ld_dw=dw.ld,
               stride_dw=dw.stride)
        want, want_w = ops.expert_linear_backward(dy, x, weight, offsets, add=add, dw_dtype=wt)
        assert torch.equal(dw.t.view(E, N, K) if E == 1 else dw.t, want_w) and dw.untouched()
        if n:
            assert torch.equal(dx.t, want) and dx.untouched()
    assert ops.status() == (0, 0)
