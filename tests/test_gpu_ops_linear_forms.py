"""Every form of a product (tests/linear_forms.py) on whole numbers: all products and sums are
exact in fp32, so a wrong, missing or doubled partial sum shows."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests.linear_forms import SHAPES  # noqa: E402
from tile_signaled_grouped_gb300 import ops  # noqa: E402


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_whole_numbers_are_exact(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    whole = lambda n, c: torch.randint(-4, 5, (n, (c + 7) // 8 * 8), generator=g,  # noqa: E731
                                       device="cuda").bfloat16()[:, :c]
    x, w, dy, r = whole(M, K), whole(N, K), whole(M, N), whole(M, N)
    b = torch.randint(-4, 5, (N,), generator=g, device="cuda").float()
    y, _ = ops.linear(x, w, out_dtype=torch.float32)
    want = x.double() @ w.double().t()
    assert torch.equal(y.double(), want)
    want += b.double()
    y, z = ops.linear(x, w, b, act="relu", residual=r, preact=True, out_dtype=torch.float32)
    assert torch.equal(z, want.bfloat16())
    assert torch.equal(y.double(), want.clamp(min=0) + r.double())

    dx, dw = (dy.double() @ w.double()).bfloat16(), dy.double().t() @ x.double()
    for need_dx, need_dw in ((True, False), (False, True), (True, True)):
        gx, gw, gb = ops.linear_backward(dy, x, w, bias=torch.float32, dw_dtype=torch.float32,
                                         need_dx=need_dx, need_dw=need_dw)
        assert (gx is not None) == need_dx and (gw is not None) == need_dw
        assert gx is None or torch.equal(gx, dx)
        assert gw is None or torch.equal(gw.double(), dw)
        assert torch.equal(gb.double(), dy.double().sum(0))
    assert ops.status() == (0, 0)
