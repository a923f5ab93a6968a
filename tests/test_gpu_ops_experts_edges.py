"""The operators on expert rows at the edges of what their documentation allows, into memory that holds NaN
before the call: what a call leaves unwritten shows."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import experts_ref as X  # noqa: E402
from tests.test_gpu_ops_experts import experts_case  # noqa: E402
from tile_signaled_grouped_gb300 import capi, ops  # noqa: E402

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
    for bad in ([-7, 40, 90, 150], [0, 40, 90, 10 ** 6], [0, 40, 40, 40], [150, 150, 150, 150], [7, 7, 10 ** 6, 10 ** 6]):
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
