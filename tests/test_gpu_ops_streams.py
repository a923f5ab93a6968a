"""The operators on two streams, and from two host threads, each with its own data: what one call
shares with another (a workspace, a partial sum, a status) would mix the two."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

from tests.test_gpu_ops_linear import mat  # noqa: E402
from tile_signaled_grouped_gb300 import ops  # noqa: E402

STEPS = 12


def work(seed, M, N, K, E):
    """A step of every operator and its backward pass on data of its own; returns step(stream)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, w, dy = mat(g, M, K, "bf16"), mat(g, N, K, "bf16", std=K ** -0.5), mat(g, M, N, "bf16")
    nw, nb = (torch.randn(K, generator=g, device="cuda") for _ in range(2))
    logits, d_w = torch.randn(M, E, generator=g, device="cuda"), torch.randn(M, 4, generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda") * 0.1

    def step(stream=None):
        h, s, mean, rstd = ops.layer_norm(x, nw, nb, residual=x, stats=True, stream=stream)
        y, z = ops.linear(h, w, act="silu", residual=dy, preact=True, stream=stream)
        dx, dw, db = ops.linear_backward(dy, h, w, z=z, act="silu", bias=torch.float32, stream=stream)
        ids, rw = ops.route_experts(logits, 4, score="sigmoid", bias=bias, renorm=True, stream=stream)
        dl = ops.route_experts_backward(d_w, logits, ids, score="sigmoid", renorm=True, stream=stream)
        return (h, s, mean, rstd, y, z, dx, dw, db, ids, rw, dl,
                *ops.layer_norm_backward(dx, s, nw, mean, rstd, dz=h, stream=stream))

    return step


@pytest.mark.parametrize("threads", [False, True], ids=["one thread", "two threads"])
@pytest.mark.parametrize("shapes", [
    [(700, 768, 1024, 64), (700, 768, 1024, 64)],      # tiles in parts, workspaces of one size
    [(2100, 1536, 2048, 128), (2100, 1536, 2048, 128)],  # CTA pairs, norms from the ring
    [(5, 517, 1000, 96), (1300, 301, 520, 33)],
], ids=str)
def test_two_streams_with_their_own_data(shapes, threads):
    steps = [work(seed, *s) for seed, s in enumerate(shapes)]
    want = []
    for step in steps:
        want.append(step())
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [[], []]
    if threads:
        start = threading.Barrier(2)

        def run(i):
            start.wait()
            for _ in range(STEPS):
                got[i].append(steps[i](streams[i]))

        both = [threading.Thread(target=run, args=(i,)) for i in range(2)]
        for t in both:
            t.start()
        for t in both:
            t.join()
    else:
        for _ in range(STEPS):
            for i in range(2):
                got[i].append(steps[i](streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == STEPS
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    assert ops.status() == (0, 0)
