"""8-bit checkpoints, bit for bit, and the gated activation with its backward pass against float64; the
backward pass of linear from checkpoints."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import experts_ref as X  # noqa: E402
from tests import ops_ref as R  # noqa: E402
from tests.test_gpu_ops_experts import gen, matrix  # noqa: E402
from tests.test_gpu_ops_linear import DT, ROUND, close  # noqa: E402
from tile_signaled_grouped_gb300 import ops  # noqa: E402

SHAPES = [(1, 1), (1, 31), (2, 32), (3, 33), (5, 64), (7, 136), (33, 1531), (16, 4096), (1, 7168), (300, 40)]


# --------------------------------------------------------------------------- checkpoints
def same_checkpoint(kept, x):
    code, unit = X.encode(x)
    got = kept.codes.double().cpu()
    scale = torch.ldexp(torch.ones(kept.scales.shape, dtype=torch.float64), kept.scales.cpu().int() - 127)
    assert torch.equal(scale, unit)
    assert torch.equal(torch.isnan(got), torch.isnan(code))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(code))
    return code, unit


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,c", SHAPES)
@pytest.mark.parametrize("pad", [0, 5, 8])
def test_checkpoint_and_restore(n, c, pad, dtype):
    g = gen(n, c)
    x = matrix(g, n, c, dtype, pad)
    # blocks of very different sizes, and elements far below their block's largest
    x = (x.float() * torch.exp2(torch.randint(-9, 9, (n, c), generator=g, device="cuda").float())).to(x.dtype)
    if pad:
        wide = torch.zeros(n, c + pad, dtype=x.dtype, device="cuda")
        wide[:, :c] = x
        x = wide[:, :c]
    kept = ops.checkpoint(x)
    assert kept.codes.shape == x.shape and kept.scales.shape == (n, -(-c // 32))
    code, unit = same_checkpoint(kept, x)
    value = X.decode(code, unit).cuda()
    for out in DT.values():
        back = ops.restore(kept, out)
        # one rounding, at most: to the nearest, ties to even, as a conversion from float64
        assert torch.equal(back, value.to(torch.float32).to(out))
    assert ((value - x.double()).abs() <= torch.maximum(
        2.0 ** -4 * x.double().abs(), 2.0 ** -10 * X.decode(torch.ones_like(code), unit).cuda())).all()


def test_checkpoint_of_special_values():
    rows = [[0.0] * 32, [-0.0] * 32, [448.0] + [0.0] * 31, [448.5] + [1.0] * 31, [1.75, -1.0], [1.7578125, 2.0 ** -9],
            [math.inf, 1.0, -3.0], [-math.inf] * 32, [math.nan, 2.0], [3.0e38, 1.0], [1e-38, 1e-40, -1e-44],
            [1e-45] * 4, [2.0 ** -120, 2.0 ** -136, 2.0 ** -137], [17.0, 19.0, 21.0, 23.0, 25.0, 27.0, 200.0]]
    x = torch.zeros(len(rows), 45, device="cuda")
    for i, r in enumerate(rows):
        x[i, :len(r)] = torch.tensor(r)
    kept = ops.checkpoint(x)
    code, unit = same_checkpoint(kept, x)
    back = ops.restore(kept, torch.float32)
    assert torch.equal(torch.nan_to_num(back), torch.nan_to_num(X.decode(code, unit)).float().cuda())
    assert torch.equal(torch.isnan(back), ~torch.isfinite(x))


def test_every_code_is_restored():
    """The 256 codes (two of them NaN) with scales from the least to the largest."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).repeat(4, 1)
    scales = torch.tensor([0, 1, 127, 246], dtype=torch.uint8, device="cuda")[:, None].repeat(1, 8)
    want = torch.ldexp(codes.double(), scales.int().repeat_interleave(32, 1) - 127).float()
    back = ops.restore(ops.Checkpoint(codes, scales), torch.float32)
    assert torch.equal(torch.isnan(back), torch.isnan(want)) and int(torch.isnan(want).sum()) == 8
    assert torch.equal(torch.nan_to_num(back), torch.nan_to_num(want))


# ----------------------------------------------------------------------- gated activation
def check_gated(gate, up, dh, act, need_h, kept):
    g, u, d = gate.double(), up.double(), dh.double()
    ea, eg = R.act_error(g, act)
    a, ag = R.act(g, act), R.act_grad(g, act)
    want_h, tol_h = a * u, ea * u.abs() + R.U32 * (a * u).abs()
    source = kept if kept is not None else (gate, up)
    dg, du, h = ops.gated_backward(dh, *source, act=act, need_h=need_h)
    rest = 3 * R.U32  # of the two products
    close(du, d * a, d.abs() * ea + rest * (d * a).abs())
    close(dg, d * u * ag, (d * u).abs() * eg + rest * (d * u * ag).abs())
    if need_h:
        close(h, want_h, tol_h)
    else:
        assert h is None
    return want_h, tol_h


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "none"])
@pytest.mark.parametrize("n,c,dtype,pad", [(1, 1, "bf16", 0), (1, 2048, "bf16", 0), (3, 33, "fp16", 5),
                                           (37, 136, "bf16", 8), (130, 1531, "fp16", 5), (64, 512, "fp16", 0),
                                           (9, 4104, "bf16", 3)])
def test_gated(n, c, dtype, pad, act):
    g = gen(n, c)
    gate, up, dh = (matrix(g, n, c, dtype, pad, std) for std in (2.0, 1.0, 1.0))
    want, tol = check_gated(gate, up, dh, act, True, None)
    h, none = ops.gated(gate, up, act=act)
    assert none is None
    close(h, want, tol)
    h8, kept = ops.gated(gate, up, act=act, checkpoint=True)
    assert torch.equal(h8, h)
    for k, x in zip(kept, (gate, up)):
        alone = ops.checkpoint(x)
        assert torch.equal(k.codes.view(torch.uint8), alone.codes.view(torch.uint8))
        assert torch.equal(k.scales, alone.scales)
    from_kept = [ops.restore(k, torch.float32) for k in kept]
    check_gated(*from_kept, dh, act, n % 2 == 1, kept)
    assert ops.status() == (0, 0)


def test_gated_columns_of_one_matrix():
    """Both halves of a product's rows, and gradients into no rows."""
    z = matrix(gen(3), 50, 2 * 264, "bf16")
    gate, up = z[:, :264], z[:, 264:]
    h, _ = ops.gated(gate, up)
    same, _ = ops.gated(gate.contiguous(), up.contiguous())
    assert torch.equal(h, same)
    empty = z[:0, :264]
    h, kept = ops.gated(empty, empty, checkpoint=True)
    assert h.shape == (0, 264) and kept[0].codes.shape == (0, 264)
    dg, du, h = ops.gated_backward(empty, *kept, need_h=True)
    assert dg.shape == du.shape == h.shape == (0, 264)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_gradient_against_differences(act):
    """h moves by dgate and dup when gate and up move: central differences in float64 of the formula at the
    kernel's inputs (fourth-order error 1e-10 at a step of 1e-3)."""
    g = gen(11)
    gate, up, dh = (matrix(g, 8, 96, "fp16") for _ in range(3))
    dg, du, _ = ops.gated_backward(dh, gate, up, act=act)
    step = 1e-3
    f = lambda v: R.act(v, act)  # noqa: E731
    x, d = gate.double(), dh.double()
    slope = (8 * (f(x + step) - f(x - step)) - (f(x + 2 * step) - f(x - 2 * step))) / (12 * step)
    tol = (d * up.double()).abs() * (R.act_error(x, act)[1] + 1e-9 + 3 * R.U32 * slope.abs())
    close(dg, d * up.double() * slope, tol)
    close(du, d * f(x), d.abs() * (R.act_error(x, act)[0] + 3 * R.U32 * f(x).abs()))


# ------------------------------------------------------------------------ linear from 8 bits
@pytest.mark.parametrize("M,N,K,dtype,act,bias", [
    (1, 8, 8, "bf16", "silu", True), (5, 40, 72, "fp16", "gelu", False), (77, 33, 64, "bf16", "silu", True),
    (300, 520, 1000, "fp16", "relu", True), (1025, 1536, 256, "bf16", "gelu_tanh", True),
    (2100, 256, 1536, "bf16", "none", True)])
def test_linear_backward_from_checkpoints(M, N, K, dtype, act, bias):
    """As from the restored matrices: the same bits for dw (x is restored for it), and, where z is read as
    it is kept, dz within the errors of act'."""
    g = gen(M, N, K)
    x, w, dy = matrix(g, M, K, dtype), matrix(g, N, K, dtype, std=K ** -0.5), matrix(g, M, N, dtype)
    z = matrix(g, M, N, dtype) if act != "none" else None
    x8, z8 = ops.checkpoint(x), None if z is None else ops.checkpoint(z)
    btype = torch.float32 if bias else None
    dx, dw, db = ops.linear_backward(dy, x8, w, z=z8, act=act, bias=btype)
    xr = ops.restore(x8, x.dtype)
    dz, edz = dy.double(), 0 * dy.double()
    if act != "none":
        zr = ops.restore(z8, torch.float32).double()
        dz = dz * R.act_grad(zr, act)
        edz = dy.double().abs() * (R.act_error(zr, act)[1] + R.U32)
    sub = 2.0 ** -25 if dtype == "fp16" else 0.0
    rounded = edz + (ROUND[x.dtype] * dz.abs() + sub if act != "none" else 0)
    w64, x64 = w.double(), xr.double()
    close(dx, dz @ w64, R.product_error(dz, w64, N) * 1.01 + rounded @ w64.abs())
    close(dw, dz.t() @ x64, R.product_error(dz.t(), x64, M) * 1.01 + rounded.t() @ x64.abs())
    if bias:
        close(db, dz.sum(0), edz.sum(0) + (M / 8 + 48 + 16) * R.U32 * dz.abs().sum(0))
    # either of the two alone
    if act == "none":
        again = ops.linear_backward(dy, xr, w, bias=btype)
        assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)) if a is not None)
    else:
        again = ops.linear_backward(dy, xr, w, z=z8, act=act, bias=btype)
        assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)) if a is not None)
        only = ops.linear_backward(dy, x8, w, z=z8, act=act, need_dw=False)
        assert torch.equal(only[0], dx) and only[1] is None
    assert ops.status() == (0, 0)


def test_linear_backward_from_checkpoints_of_no_rows():
    none = ops.checkpoint(torch.empty(0, 24, device="cuda").bfloat16())
    dy, w = torch.empty(0, 16, device="cuda").bfloat16(), torch.ones(16, 24, device="cuda").bfloat16()
    dx, dw, db = ops.linear_backward(dy, none, w, z=ops.checkpoint(dy), act="silu", bias=torch.float32)
    assert dx.shape == (0, 24) and not dw.any() and not db.any()
    assert ops.restore(none, torch.float16).shape == (0, 24)
