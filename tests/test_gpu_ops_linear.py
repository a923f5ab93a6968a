"""The matrix product with its epilogue (ops.linear and its backward) against float64,
within the rounding errors of the operands' types and of fp32 sums."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import ops_ref as R  # noqa: E402
from tile_signaled_grouped_gb300 import ops  # noqa: E402

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}

# M, N, K, dtype, act, btype, residual, out, pad
CASES = [
    (1, 1, 1, "bf16", "none", None, False, None, 0),
    (1, 2048, 7168, "bf16", "silu", "fp32", False, None, 0),
    (1, 256, 7168, "bf16", "none", None, False, "fp32", 0),
    (2, 8, 2048, "fp16", "none", "fp16", True, "fp32", 8),
    (3, 517, 72, "fp16", "gelu", "fp16", True, None, 8),
    (8, 1536, 4096, "bf16", "gelu_tanh", "bf16", True, None, 0),
    (9, 130, 260, "bf16", "relu", "fp32", False, None, 4),
    (16, 4096, 1536, "bf16", "silu", None, True, None, 0),
    (17, 33, 64, "fp16", "none", "fp32", True, None, 0),
    (32, 2048, 2048, "fp16", "silu", "fp32", False, None, 0),
    (33, 300, 1000, "bf16", "gelu", "bf16", True, None, 0),
    (64, 7168, 256, "bf16", "none", "fp32", True, None, 0),
    (100, 129, 65, "bf16", "none", None, False, None, 7),
    (128, 128, 128, "bf16", "none", None, False, "fp32", 0),
    (200, 1000, 4096, "fp16", "relu", "fp32", True, "fp32", 0),
    (256, 256, 2048, "bf16", "none", "bf16", False, None, 0),
    (333, 517, 1000, "fp16", "gelu", "fp16", True, None, 8),
    (1000, 2056, 520, "bf16", "gelu_tanh", "fp32", True, None, 0),
    (2048, 1536, 4096, "bf16", "none", None, False, None, 0),
    (4097, 2049, 192, "bf16", "silu", "fp32", True, None, 0),
    (3000, 5120, 100, "fp16", "none", "fp32", False, None, 4),
]


def mat(g, n, c, dtype, pad=0, std=1.0):
    """Random [n, c] inside rows of a multiple of 8 elements, `pad` rounded up to it wider."""
    wide = (c + pad + 7) // 8 * 8
    t = torch.randn(n, wide, generator=g, device="cuda") * std
    return t.to(DT[dtype])[:, :c]


def close(got, want, tol):
    rnd = ROUND[got.dtype] * (want.abs() + tol)
    if got.dtype == torch.float16:
        rnd = rnd.clamp(min=2.0 ** -25)
    err = (got.double() - want).abs()
    bad = ~(err <= tol + rnd + 1e-37)
    assert not bad.any(), (int(bad.sum()), float((err / (tol + rnd + 1e-37)).max()))


def check(x, w, b, r, act, out, dy, seed=0):
    y, z = ops.linear(x, w, b, act=act, residual=r, preact=True, out_dtype=out)
    assert y.dtype == (out or x.dtype) and z.dtype == x.dtype
    x64, w64 = x.double(), w.double()
    zw = x64 @ w64.t()
    tz = R.product_error(x64, w64.t(), x.shape[1])
    if b is not None:
        zw = zw + b.double()
        tz = tz + R.U32 * zw.abs()
    close(z, zw, tz)
    ea, _ = R.act_error(zw, act)
    yw, ty = R.act(zw, act), 1.13 * tz + ea
    if r is not None:
        yw = yw + r.double()
        ty = ty + R.U32 * (yw.abs() + ty)
    close(y, yw, ty)
    y2, none = ops.linear(x, w, b, act=act, residual=r, out_dtype=out)
    assert none is None and torch.equal(y2, y)

    # Backward from the stored z. With an activation the products' dz is rounded.
    btype = None if b is None else b.dtype
    zb = z if act != "none" else None
    dx, dw, db = ops.linear_backward(dy, x, w, z=zb, act=act, bias=btype,
                                     dw_dtype=torch.float32 if out == torch.float32 else None)
    dz, edz = dy.double(), 0 * dy.double()
    if act != "none":
        z64 = z.double()
        dz = dy.double() * R.act_grad(z64, act)
        edz = dy.double().abs() * (R.act_error(z64, act)[1] + R.U32)
    sub = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    rounded = edz + (ROUND[x.dtype] * dz.abs() + sub if act != "none" else 0)
    M, N = dy.shape
    close(dx, dz @ w64, R.product_error(dz, w64, N) * 1.01 + rounded @ w64.abs())
    close(dw, dz.t() @ x64, R.product_error(dz.t(), x64, M) * 1.01 + rounded.t() @ x64.abs())
    if btype is not None:
        # M / 8 rows of a warp at most (ranges of eight rows or more), eight warps, 256 ranges
        close(db, dz.sum(0), edz.sum(0) + (M / 8 + 48 + 16) * R.U32 * dz.abs().sum(0))
    assert ops.status() == (0, 0)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_linear(case):
    M, N, K, dtype, act, btype, residual, out, pad = case
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x, w = mat(g, M, K, dtype, pad), mat(g, N, K, dtype, pad, std=K ** -0.5)
    b = (torch.randn(N, generator=g, device="cuda") * 0.3).to(DT[btype]) if btype else None
    r = mat(g, M, N, dtype, pad) if residual else None
    dy = mat(g, M, N, dtype, pad)
    if pad == 4:
        dy = dy.contiguous()  # rows of any length: not on 16 bytes
    check(x, w, b, r, act, DT[out] if out else None, dy)


@pytest.mark.parametrize("M,N,K", [(1, 24, 8), (5, 64, 200), (70, 90, 128), (300, 700, 96),
                                   (2304, 1536, 2056), (4100, 1030, 776), (700, 5000, 3000),
                                   (6000, 300, 2500)])
def test_whole_numbers_are_exact(M, N, K):
    """Small integers: every product and sum is exact in fp32, so the fp32 results are too.
    A wrong, missing or doubled element shows."""
    g = torch.Generator(device="cuda").manual_seed(M)
    i = lambda n, c: torch.randint(-4, 5, (n, (c + 7) // 8 * 8), generator=g,  # noqa: E731
                                   device="cuda").bfloat16()[:, :c]
    x, w, dy = i(M, K), i(N, K), i(M, N)
    y, _ = ops.linear(x, w, out_dtype=torch.float32)
    assert torch.equal(y.double(), x.double() @ w.double().t())
    dx, dw, db = ops.linear_backward(dy, x, w, bias=torch.float32, dw_dtype=torch.float32)
    assert torch.equal(dw.double(), dy.double().t() @ x.double())
    assert torch.equal(db.double(), dy.double().sum(0))
    assert torch.equal(dx, (dy.double() @ w.double()).bfloat16())


def test_bad_values_stay_in_their_rows_and_columns():
    g = torch.Generator(device="cuda").manual_seed(1)
    for M in (20, 200):
        x, w = mat(g, M, 136, "bf16").clone(), mat(g, 200, 136, "bf16").clone()
        want, _ = ops.linear(x, w, act="relu")
        x[7, 5], w[9, 130] = float("nan"), float("inf")
        y, _ = ops.linear(x, w, act="relu")
        keep = torch.ones_like(y, dtype=torch.bool)
        keep[7], keep[:, 9] = False, False
        assert torch.equal(y[keep], want[keep])
        assert torch.isnan(y[7]).all()
        assert (~torch.isfinite(y[:, 9]) | (y[:, 9] == 0)).all()  # act(-inf) is 0


def test_extreme_activations():
    """act and act' of 0, of the largest values and of infinities."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3.0, -3.0, 30.0, -30.0, 1e4, -1e4, 3e38, -3e38],
                     device="cuda").bfloat16()[None]
    one = torch.ones(1, 12, device="cuda").bfloat16()
    x, w = torch.ones(1, 8, device="cuda").bfloat16(), torch.zeros(12, 8, device="cuda").bfloat16()
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        w[:, 0] = z[0]
        y, _ = ops.linear(x, w, act=act)
        want = R.act(z.double(), act)
        want = torch.where(z.double() < -1e3, torch.zeros_like(want), want)
        want = torch.where(z.double() > 1e3, z.double(), want)
        assert (y.double() - want).abs().le(2.0 ** -8 * want.abs() + 1e-6).all(), act
        _, _, db = ops.linear_backward(one, x, w, z=z, act=act, bias=torch.float32)
        want = R.act_grad(z.double().clamp(-40, 40), act)
        assert (db.double() - want[0]).abs().max() < 1e-5, act


def test_empty_one_dimension_and_more():
    w = torch.randn(24, 16, device="cuda").bfloat16()
    x0 = torch.zeros(0, 16, device="cuda").bfloat16()
    y, z = ops.linear(x0, w, preact=True)
    assert y.shape == (0, 24) and z.shape == (0, 24)
    dx, dw, db = ops.linear_backward(y, x0, w, bias=torch.float32)
    assert dx.shape == (0, 16) and dw.shape == (24, 16) and not dw.any() and not db.any()
    x = torch.randn(2, 3, 16, device="cuda").bfloat16()
    y3, _ = ops.linear(x, w)
    assert y3.shape == (2, 3, 24)
    assert torch.equal(y3.view(6, 24), ops.linear(x.view(6, 16), w)[0])
    assert ops.linear(x[0, 0], w)[0].shape == (24,)
    dx, dw, _ = ops.linear_backward(y3, x, w)
    assert dx.shape == x.shape
    assert ops.linear_backward(y3, x, w, need_dx=False)[0] is None
    assert ops.linear_backward(y3, x, w, need_dw=False)[1] is None


def test_rows_past_32_bit_offsets():
    """Row 519 of x, of the residual and of dy lies 2.2e9 elements from the first."""
    ld, n, c = 1 << 22, 520, 64
    big = torch.empty((n - 1) * ld + c, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((n, c), (ld, 1))
    g = torch.Generator(device="cuda").manual_seed(2)
    src, w = mat(g, n, c, "bf16"), mat(g, c, c, "bf16")
    x.copy_(src)
    assert torch.equal(ops.linear(x, w, residual=x)[0], ops.linear(src, w, residual=src)[0])
    a = ops.linear_backward(x, x, w, z=x, act="silu", bias=torch.float32)
    b = ops.linear_backward(src, src, w, z=src, act="silu", bias=torch.float32)
    c = ops.linear_backward(x, x, w)
    d = ops.linear_backward(src, src, w)
    for p, q in zip(a + c[:2], b + d[:2]):
        assert torch.equal(p, q)


def test_repeats_streams_and_graphs_give_the_same_bits():
    g = torch.Generator(device="cuda").manual_seed(3)
    for M in (4, 60, 700, 2100):
        x, w, dy = mat(g, M, 1024, "bf16"), mat(g, 768, 1024, "bf16"), mat(g, M, 768, "bf16")

        def step(stream=None):
            y, z = ops.linear(x, w, act="silu", residual=dy, preact=True, stream=stream)
            return (y, z, *ops.linear_backward(dy, x, w, z=z, act="silu", bias=torch.float32,
                                               stream=stream))

        want = step()
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        for got in (step(), step(st)):
            st.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        x.copy_(mat(g, M, 1024, "bf16"))
        graph.replay()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    ops.clear_status()
    assert ops.status() == (0, 0)


# gelu(z) = z Phi(z), Phi(z) = erfc(-z / sqrt(2)) / 2. In fp32, relative to Phi and in half steps: three
# roundings of the exponent -z^2 / 2 (1.5 z^2), the exponential and the reciprocal (4 each, and 2 for the
# latter's argument), 8 terms of a fit and its own error (12), products (3).
def gelu_steps(z):
    return 1.5 * z * z + 28


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [1, 20])
def test_gelu_keeps_its_relative_accuracy_below_zero(M, dtype):
    z = torch.linspace(-9.0, 3.0, 769, device="cuda").to(DT[dtype])
    x = torch.zeros(M, 8, device="cuda", dtype=DT[dtype])
    x[:, 0] = 1
    w = torch.zeros(z.numel(), 8, device="cuda", dtype=DT[dtype])
    w[:, 0] = z
    z = z.double()
    want = R.act(z, "gelu")
    tol = gelu_steps(z) * R.U32 * want.abs()
    y, _ = ops.linear(x, w, act="gelu", out_dtype=torch.float32)
    assert ((y.double() - want).abs() <= tol).all()
    y, _ = ops.linear(x, w, act="gelu")
    tol = tol + ROUND[y.dtype] * want.abs() + (2.0 ** -25 if dtype == "fp16" else 0.0)
    assert ((y.double() - want).abs() <= tol).all()


def test_gelu_gradient_below_zero():
    """gelu' = Phi + z phi: each term to its relative error."""
    z = torch.linspace(-9.0, 3.0, 769, device="cuda").bfloat16()[None]
    x, w = torch.zeros(1, 8, device="cuda").bfloat16(), torch.zeros(769, 8, device="cuda").bfloat16()
    _, _, db = ops.linear_backward(torch.ones_like(z), x, w, z=z, act="gelu", bias=torch.float32)
    z = z[0].double()
    cdf = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    pdf = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    tol = gelu_steps(z) * R.U32 * (cdf + (z * pdf).abs())
    assert ((db.double() - R.act_grad(z, "gelu")).abs() <= tol).all()


def test_silu_gradient_far_below_zero():
    """silu'(z) = q (1 + z (1 - q)), relative to itself, in half steps: the exponential 4 + 2.4 |z|,
    the division 4, the sums and products around them 7. Below the range of fp32 it is 0."""
    z = torch.tensor([-20.0, -29.5, -30.0, -31.0, -45.0, -60.0, -85.0, -100.0, -1e4, -3e38, -math.inf],
                     device="cuda").bfloat16()[None]
    x, w = torch.zeros(1, 8, device="cuda").bfloat16(), torch.zeros(11, 8, device="cuda").bfloat16()
    _, _, db = ops.linear_backward(torch.ones_like(z), x, w, z=z, act="silu", bias=torch.float32)
    z = z[0, :7].double()
    want = R.act_grad(z, "silu")
    assert ((db[:7].double() - want).abs() <= (2.4 * z.abs() + 16) * R.U32 * want.abs()).all()
    assert not db[7:].any()
