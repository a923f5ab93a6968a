"""One feed-forward half of a transformer block on one GPU: norm, router, routed experts and
a dense expert (block.MoEBlock), first for a prompt, then a training step, and the routed experts
alone for a few tokens (block.Experts).

    python examples/moe_block.py [workload]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tile_signaled_grouped_gb300 import ops  # noqa: E402
from tile_signaled_grouped_gb300.block import Experts, MoEBlock  # noqa: E402
from tile_signaled_grouped_gb300.runtime import ExpertCombine  # noqa: E402
from tile_signaled_grouped_gb300.workloads import get_workload, make_inputs  # noqa: E402


def main(name="tiny"):
    torch.manual_seed(0)
    wl = get_workload(name)
    inp = make_inputs(wl, device="cuda")
    d, hidden = wl.d_model, wl.d_ff
    layer = ExpertCombine(wl.W, wl.L, wl.topk, wl.T, d, wl.d_ff, wl.tb_M)
    router = ops.router_cfg(wl.E, wl.topk, score="sigmoid", renorm=True, scale=2.5)
    normal = lambda *shape, std: (torch.randn(*shape, device="cuda") * std).bfloat16()  # noqa: E731
    experts = Experts(*(torch.cat(list(w)) for w in (inp.w_gate, inp.w_up, inp.w_down)))
    w_gate, w_up, w_down = experts.ranks(wl.W)  # the layer's lists: the same memory
    block = MoEBlock(layer, router, norm_w=1 + normal(d, std=0.1), norm_b=normal(d, std=0.1),
                     w_router=normal(wl.E, d, std=d ** -0.5), w1=normal(hidden, d, std=d ** -0.5),
                     b1=torch.zeros(hidden, device="cuda"), w2=normal(d, hidden, std=hidden ** -0.5),
                     b2=torch.zeros(d, device="cuda"), w_gate=w_gate, w_up=w_up,
                     w_down=w_down, router_bias=torch.zeros(wl.E, device="cuda"), experts=experts)
    x = torch.cat(list(inp.x))
    torch.cuda.synchronize()

    y, moe, _ = block.forward(x)  # the next block takes y as x and moe as residual
    y, moe, _ = block.forward(y, residual=moe)
    torch.cuda.synchronize()
    print(f"{name}: {x.shape[0]} tokens, two blocks; output norm {float((y + moe).float().norm()):.1f}, "
          f"status {layer.status()}, {ops.status()}")

    y, moe, saved = block.forward(x, save=True)
    grads = block.backward(torch.ones_like(y), saved, d_moe=torch.ones_like(moe))
    torch.cuda.synchronize()
    print("gradient norms:", {k: round(float(v.float().norm()), 2) for k, v in grads.items()})

    few = saved["h"][:3]  # any number of tokens: no plan, no ranks
    ids, w = ops.route_experts(saved["logits"][:3], wl.topk, score="sigmoid", renorm=True, scale=2.5)
    out, _ = experts.forward(few, ids, w)
    torch.cuda.synchronize()
    print(f"experts of 3 tokens: norm {float(out.float().norm()):.2f}, status {ops.status()}")
    layer.close()


if __name__ == "__main__":
    main(*sys.argv[1:2])
