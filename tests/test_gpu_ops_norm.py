"""Layer norm (ops.layer_norm and its backward) against float64, within the rounding errors
of their formulas."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import ops_ref as R  # noqa: E402
from tile_signaled_grouped_gb300 import ops  # noqa: E402

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
EPS = 1e-5

# n, D, dtype, wtype, residual, weight, bias, pad
CASES = [
    (1, 7168, "bf16", "bf16", True, True, True, 0),
    (3, 1531, "fp16", "fp32", False, True, False, 5),
    (700, 128, "bf16", "fp32", True, True, True, 0),
    (65, 41, "fp32", "fp32", True, True, True, 3),
    (400, 4096, "bf16", "bf16", True, True, True, 8),
    (320, 5120, "fp16", "fp16", False, True, True, 0),
    (310, 8192, "bf16", "fp32", True, False, True, 0),
    (5, 8192, "fp32", "fp32", False, True, True, 0),
    (306, 7167, "fp32", "fp32", True, True, True, 0),
    (306, 9000, "bf16", "bf16", False, True, True, 0),
    (2, 16384, "fp16", "fp32", False, False, False, 0),
    (307, 16383, "bf16", "fp32", True, True, True, 1),
    (2, 20000, "fp32", "fp32", True, True, True, 0),
    (7, 33001, "bf16", "bf16", True, True, True, 2),
    (1, 1, "fp32", "fp32", False, True, True, 0),
    (9, 2, "bf16", "bf16", True, True, True, 6),
    (2000, 264, "fp16", "fp16", True, True, True, 0),
    # rows from the ring of shared memory
    (1300, 4096, "bf16", "fp32", True, True, True, 0),
    (1217, 520, "fp16", "fp16", False, True, False, 8),
    (700, 7168, "bf16", "bf16", True, True, True, 16),
    (640, 8192, "fp32", "fp32", True, True, True, 0),
    (1500, 1032, "fp32", "fp32", False, False, True, 4),
    # and rows that start anywhere
    (1300, 4097, "bf16", "fp32", True, True, True, 0),
    (1250, 1531, "fp16", "fp16", True, True, True, 5),
    (700, 5003, "fp32", "fp32", True, True, False, 3),
    (640, 8191, "bf16", "bf16", False, True, True, 1),
    (4900, 37, "fp32", "fp32", True, False, True, 2),
    (4900, 301, "bf16", "bf16", True, True, True, 0),
    (2700, 1024, "fp16", "fp32", True, True, True, 5),
]


def rows(g, n, D, dtype, pad, mean=0.3):
    t = torch.randn(n, D + pad, generator=g) * 1.3 + mean
    return t.to(DT[dtype]).cuda()[:, :D]


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, tol):
    """Within tol and the rounding to got's type."""
    rnd = ROUND[got.dtype] * (np.abs(want) + tol)
    if got.dtype == torch.float16:
        rnd = np.maximum(rnd, 2.0 ** -25)
    bad = ~(np.abs(np64(got) - want) <= tol + rnd + 1e-37)
    assert not bad.any(), (np.abs(np64(got) - want)[bad].max(), bad.sum())


def check(x, w, b, r, dy, dz, eps=EPS):
    y, z, mean, rstd = ops.layer_norm(x, w, b, eps=eps, residual=r, stats=True)
    want = R.layer_norm(np64(x), np64(w), np64(b), eps, np64(r))
    tol = R.layer_norm_tolerance(np64(x), np64(w), np64(b), eps, np64(r))
    for got, e, t in zip((y, z, mean, rstd), want, tol):
        close(got, e, t)
    assert (z is x) == (r is None)
    for flag in (True, False):
        dx, dw, db = ops.layer_norm_backward(dy, z, w, mean, rstd, dz=dz, bias=flag)
        args = (np64(dy), np64(z), np64(w), np64(mean), np64(rstd), np64(dz))
        want, tol = R.layer_norm_backward(*args), R.layer_norm_backward_tolerance(*args)
        close(dx, want[0], tol[0])
        assert (dw is None) == (w is None) and (db is not None) == flag
        if dw is not None:
            assert dw.dtype == w.dtype
            close(dw, want[1], tol[1])
        if flag:
            close(db, want[2], tol[2])


@pytest.mark.parametrize("case", CASES, ids=str)
def test_layer_norm(case):
    n, D, dtype, wtype, residual, weight, bias, pad = case
    g = torch.Generator().manual_seed(n + D)
    x = rows(g, n, D, dtype, pad)
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(DT[wtype]).cuda() if weight else None
    b = (0.3 * torch.randn(D, generator=g)).to(DT[wtype]).cuda() if bias else None
    r = rows(g, n, D, dtype, 2 * pad, 0.0) if residual else None
    check(x, w, b, r, rows(g, n, D, dtype, pad, 0.0), rows(g, n, D, dtype, 0, 0.0) if residual else None)


def test_flat_rows_and_large_offsets():
    """A row of one value has variance 0 (y = b); one far from zero keeps its variance."""
    g = torch.Generator().manual_seed(1)
    x = rows(g, 12, 1000, "fp32", 0)
    x[3] = 7.25
    x[4] = 0.0
    x[5] += 3000.0
    w, b = torch.randn(1000, generator=g).cuda(), torch.randn(1000, generator=g).cuda()
    check(x, w, b, None, rows(g, 12, 1000, "fp32", 0), None)
    y = ops.layer_norm(x, w, b)[0]
    assert torch.equal(y[3], b) and torch.equal(y[4], b)


def test_a_bad_row_stays_alone():
    g = torch.Generator().manual_seed(2)
    x = rows(g, 9, 300, "bf16", 0)
    w = torch.ones(300, device="cuda", dtype=torch.bfloat16)
    want, _, wm, wr = ops.layer_norm(x, w, stats=True)
    x2 = x.clone()
    x2[4, 7] = float("nan")
    x2[6, 0] = float("inf")
    y, _, mean, rstd = ops.layer_norm(x2, w, stats=True)
    ok = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[ok], want[ok]) and torch.equal(mean[ok], wm[ok])
    assert torch.isnan(y[4]).all() and torch.isnan(y[6]).all()
    dx, _, _ = ops.layer_norm_backward(want, x2, w, mean, rstd)
    wx, _, _ = ops.layer_norm_backward(want, x, w, wm, wr)
    assert torch.equal(dx[ok], wx[ok])


def test_empty_one_dimension_and_more():
    w = torch.ones(16, device="cuda")
    y, z, mean, rstd = ops.layer_norm(torch.zeros(0, 16, device="cuda"), w, stats=True)
    assert y.shape == (0, 16) and mean.shape == (0,)
    dx, dw, db = ops.layer_norm_backward(y, z, w, mean, rstd)
    assert dx.shape == (0, 16) and not dw.any() and not db.any()
    x = torch.randn(2, 3, 16, device="cuda")
    y3 = ops.layer_norm(x, w)[0]
    assert torch.equal(y3.view(6, 16), ops.layer_norm(x.view(6, 16), w)[0])
    assert torch.equal(ops.layer_norm(x[0, 0], w)[0], y3[0, 0])


def test_unaligned_bases():
    g = torch.Generator().manual_seed(3)
    for dtype in ("bf16", "fp32"):
        wide = rows(g, 40, 272, dtype, 0)
        x, dy = wide[:, 1:257], wide[:, 3:259]
        w = rows(g, 1, 257, dtype, 0)[0][1:]
        check(x, w, w, dy, dy, x)


def test_rows_past_32_bit_offsets():
    """Row 519 of x lies 2.2e9 elements from its start."""
    ld, n, D = 1 << 22, 520, 64
    big = torch.empty((n - 1) * ld + D, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((n, D), (ld, 1))
    g = torch.Generator().manual_seed(4)
    src = rows(g, n, D, "bf16", 0)
    x.copy_(src)
    w = torch.ones(D, device="cuda")
    want = ops.layer_norm(src, w, residual=src, stats=True)
    got = ops.layer_norm(x, w, residual=x, stats=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    a = ops.layer_norm_backward(x, x, w, want[2], want[3], dz=x)
    b = ops.layer_norm_backward(src, src, w, want[2], want[3], dz=src)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_repeats_streams_and_graphs_give_the_same_bits():
    g = torch.Generator().manual_seed(5)
    x, dy = rows(g, 900, 2048, "bf16", 0), rows(g, 900, 2048, "bf16", 0)
    w = torch.randn(2048, generator=g).cuda()

    def step(stream=None):
        y, z, mean, rstd = ops.layer_norm(x, w, w, residual=dy, stats=True, stream=stream)
        return (y, z, mean, rstd, *ops.layer_norm_backward(dy, z, w, mean, rstd, dz=y, stream=stream))

    want = step()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for got in (step(), step(st)):
        st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(rows(g, 900, 2048, "bf16", 0))
    graph.replay()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("n,D,dtype,pad", [(20000, 512, "bf16", 0), (20000, 301, "fp16", 3),
                                           (12000, 256, "fp32", 0)])
def test_one_warp_rows_lap_their_ring(n, D, dtype, pad):
    """Rows that one warp holds, eight and more laps of the ring's stages: a stage may take its
    next row only once every lane has read this one, the residual's gradient too."""
    g = torch.Generator().manual_seed(n + D)
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(DT[dtype]).cuda()
    check(rows(g, n, D, dtype, pad), w, w, rows(g, n, D, dtype, 0, 0.0), rows(g, n, D, dtype, pad, 0.0),
          rows(g, n, D, dtype, pad, 0.0))
