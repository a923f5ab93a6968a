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
