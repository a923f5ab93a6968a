"""What the operators on expert rows, checkpoints and the gated activation refuse, in C and on torch
tensors, and their float64 references' gradients against differences; no GPU."""
import ctypes

import pytest
import torch

from tests import experts_ref as X
from tests import ops_ref as R
from tile_signaled_grouped_gb300 import build as B

B.build()
from tile_signaled_grouped_gb300 import capi, ops  # noqa: E402
from tile_signaled_grouped_gb300.block import Experts  # noqa: E402

ARG, WORKSPACE = capi.MOE_ERR_ARG, capi.MOE_ERR_WORKSPACE


def args(cls, **kw):
    a = cls()
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def test_sort_refuses():
    f = capi.lib().moe_sort_experts
    ok = dict(ids=64, n=10, E=4, slots=64, rows=64, offsets=64, work=None, size=0)
    for bad in (dict(n=-1), dict(n=1 << 31), dict(E=0), dict(E=1025), dict(ids=None), dict(ids=2), dict(slots=None),
                dict(slots=66), dict(rows=None), dict(rows=65), dict(offsets=None), dict(offsets=66),
                dict(n=100000, work=None), dict(n=100000, work=72, size=1 << 20)):
        assert f(*{**ok, **bad}.values(), None) == ARG, bad
    need = capi.lib().moe_sort_experts_workspace(100000, 4)
    assert need > 0 and f(64, 100000, 4, 64, 64, 64, 64, need - 1, None) == WORKSPACE
    size = capi.lib().moe_sort_experts_workspace
    assert size(0, 4) == size(-1, 4) == size(10, 0) == size(10, 1025) == size(2048, 1024) == 0
    # at most 148 chunks of counts, however many slots
    assert max(size(n, 256) for n in (2049, 10 ** 6, 1 << 29)) <= 148 * 256 * 4


ROWS = dict(T=5, D=16, topk=2, E=4, dtype=capi.MOE_BF16, rows=64, offsets=64, w=64, x=64, y=64, r=64, dr=64, dw=64,
            ld_x=16, ld_y=16, ld_r=16, ld_dr=16)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=1 << 30, topk=32), dict(topk=0), dict(topk=33), dict(E=0),
                                 dict(E=1025), dict(D=0), dict(D=1 << 31), dict(dtype=3), dict(rows=None),
                                 dict(rows=66), dict(offsets=None), dict(offsets=65)], ids=str)
def test_rows_refuse(bad):
    lib = capi.lib()
    for f in (lib.moe_expert_rows, lib.moe_combine_experts, lib.moe_combine_experts_backward):
        assert f(args(capi.moe_rows_args, **{**ROWS, **bad}), None) == ARG
    assert lib.moe_expert_rows(None, None) == ARG


def test_rows_refuse_their_matrices():
    lib = capi.lib()
    for f, names in ((lib.moe_expert_rows, ("x", "dr")), (lib.moe_combine_experts, ("y", "r")),
                     (lib.moe_combine_experts_backward, ("x", "r", "dr"))):
        for k in names:
            for bad in ({k: None}, {k: 65}, {"ld_" + k: 15}, {"ld_" + k: 1 << 32}):
                assert f(args(capi.moe_rows_args, **{**ROWS, **bad}), None) == ARG, (k, bad)
        assert f(args(capi.moe_rows_args, T=0, D=16, topk=2, E=4), None) == 0
    back = lib.moe_combine_experts_backward
    for bad in (dict(w=None), dict(w=66), dict(dw=None), dict(dw=65), dict(r_scales=64, ld_scales=0)):
        assert back(args(capi.moe_rows_args, **{**ROWS, **bad}), None) == ARG, bad
    assert lib.moe_combine_experts(args(capi.moe_rows_args, **{**ROWS, "w": 66}), None) == ARG


def test_checkpoint_and_restore_refuse():
    lib = capi.lib()
    ok = dict(n=3, c=40, dtype=capi.MOE_FP16, x=64, codes=64, scales=64, ld_x=40, ld_codes=40, ld_scales=2)
    for f in (lib.moe_checkpoint, lib.moe_restore):
        for bad in (dict(n=-1), dict(c=0), dict(n=1 << 31), dict(c=1 << 31), dict(dtype=-1), dict(x=None), dict(x=65),
                    dict(codes=None), dict(scales=None), dict(ld_x=39), dict(ld_codes=39), dict(ld_scales=1)):
            assert f(args(capi.moe_checkpoint_args, **{**ok, **bad}), None) == ARG, bad
        assert f(None, None) == ARG
        assert f(args(capi.moe_checkpoint_args, **{**ok, "n": 0, "x": None}), None) == 0


def test_gated_refuses():
    lib = capi.lib()
    ok = dict(n=3, c=40, dtype=capi.MOE_BF16, act=capi.MOE_ACT_SILU, gate=64, up=64, h=64, dh=64, dgate=64, dup=64,
              ld_gate=40, ld_up=40, ld_h=40, ld_dh=40, ld_dgate=40, ld_dup=40)
    both = (dict(n=-1), dict(c=0), dict(dtype=capi.MOE_FP32), dict(act=-1), dict(act=5), dict(gate=None), dict(gate=65),
            dict(up=None), dict(ld_gate=39), dict(ld_up=39), dict(ld_h=39), dict(h=65), dict(gate_scales=64),
            dict(up_scales=64))
    for bad in both + (dict(h=None), dict(gate_codes=64), dict(gate_scales=64, up_scales=64),
                       dict(gate_scales=64, up_scales=64, gate_codes=64)):
        assert lib.moe_gated(args(capi.moe_gated_args, **{**ok, **bad}), None) == ARG, bad
    for bad in both + (dict(dh=None), dict(dgate=None), dict(dup=65), dict(ld_dh=39), dict(ld_dgate=39), dict(ld_dup=39)):
        assert lib.moe_gated_backward(args(capi.moe_gated_args, **{**ok, **bad}), None) == ARG, bad
    assert lib.moe_gated(None, None) == lib.moe_gated_backward(None, None) == ARG


def test_expert_products_refuse():
    lib = capi.lib()
    ok = dict(n=5, N=16, K=24, E=3, dtype=capi.MOE_BF16, dwtype=capi.MOE_BF16, offsets=64, x=64, w=64, y=64, dy=64,
              dx=64, dw=64, ld_x=24, ld_w=24, stride_w=384, ld_y=16, ld_dy=16, ld_add=24, ld_dx=24, ld_dw=24,
              stride_dw=384)
    both = (dict(n=-1), dict(n=1 << 31), dict(N=0), dict(N=12), dict(K=4), dict(K=20), dict(E=0), dict(E=1025),
            dict(dtype=capi.MOE_FP32), dict(offsets=None), dict(offsets=66), dict(w=None), dict(w=72), dict(ld_w=16),
            dict(ld_w=28), dict(stride_w=376), dict(stride_w=388), dict(x=None), dict(x=72), dict(ld_x=28), dict(ld_x=16))
    for bad in both + (dict(y=None), dict(y=72), dict(ld_y=8), dict(ld_y=20)):
        assert lib.moe_expert_linear(args(capi.moe_expert_linear_args, **{**ok, **bad}), None, 0, None) == ARG, bad
    for bad in both + (dict(dwtype=capi.MOE_FP16), dict(dy=None), dict(dy=72), dict(ld_dy=8), dict(dx=72), dict(ld_dx=20),
                       dict(dw=72), dict(ld_dw=28), dict(stride_dw=380), dict(add=72), dict(add=64, ld_add=16), dict(add=64, ld_add=28)):
        assert lib.moe_expert_linear_backward(args(capi.moe_expert_linear_args, **{**ok, **bad}), None, 0, None) == ARG, bad
    assert lib.moe_expert_linear(args(capi.moe_expert_linear_args, **{**ok, "n": 0, "x": None}), None, 0, None) == 0
    assert lib.moe_expert_linear_backward(args(capi.moe_expert_linear_args, **{**ok, "n": 0, "dw": None}), None, 0,
                                          None) == 0
    # a long sum over few rows is shared out: parts of 4 bytes an element, up to eight
    size = lib.moe_expert_linear_workspace
    assert size(5, 16, 24, 3) == size(0, 16, 8192, 3) == size(8, 2048, 7168, 64) == 0
    assert size(2, 256, 7168, 64) == 8 * 2 * 256 * 4 and size(5, 512, 2048, 3) == 4 * 5 * 512 * 4
    need = size(5, 16, 8192, 3)
    wide = {**ok, "K": 8192, "ld_x": 8192, "ld_w": 8192, "stride_w": 8192 * 16}
    tall = {**ok, "N": 8192, "K": 16, "ld_y": 8192, "ld_dy": 8192, "stride_w": 24 * 8192, "dw": None}
    for call, a in ((lib.moe_expert_linear, wide), (lib.moe_expert_linear_backward, tall)):
        a = args(capi.moe_expert_linear_args, **a)
        assert call(a, None, need, None) == call(a, 72, need, None) == ARG
        assert call(a, 64, need - 1, None) == WORKSPACE


def test_linear_refuses_checkpoints():
    lib = capi.lib()
    ok = dict(M=5, N=16, K=24, dtype=capi.MOE_BF16, ytype=capi.MOE_BF16, btype=capi.MOE_BF16, dwtype=capi.MOE_BF16,
              act=capi.MOE_ACT_SILU, x=64, w=64, z=64, dy=64, dx=64, dw=64, db=64, ld_x=24, ld_w=24, ld_z=16, ld_dy=16,
              ld_dx=24, ld_dw=24, z_scales=64, x_scales=64)
    size = lib.moe_linear_workspace(5, 16) + lib.moe_linear_kept_bytes(5, 24)
    f = lambda n, **bad: lib.moe_linear_backward(  # noqa: E731
        args(capi.moe_linear_args, **{**ok, **bad}), 256, n, None)
    for bad in (dict(z=None), dict(ld_z=15), dict(act=capi.MOE_ACT_NONE), dict(x=None), dict(x=68), dict(K=20)):
        assert f(size, **bad) == ARG, bad
    assert f(size - 1) == WORKSPACE
    assert lib.moe_linear_kept_bytes(5, 24) == 5 * 24 * 2 and lib.moe_linear_kept_bytes(0, 24) == 0


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def refuses(match, f, *a, **k):
    with pytest.raises(ValueError, match=match):
        f(*a, **k)


def test_tensors_are_refused():
    ids = i32(4, 2)
    refuses("ids", ops.sort_experts, ids.long(), 8)
    refuses("ids", ops.sort_experts, i32(2, 4).t(), 8)
    refuses("E is", ops.sort_experts, ids, 0)
    refuses("E is", ops.sort_experts, ids, 1025)
    refuses("CUDA", ops.sort_experts, ids, 8)
    order = ops.ExpertOrder(i32(8), i32(4, 2), i32(9))
    refuses("CUDA", ops.expert_rows, bf(4, 16), order)
    refuses("order", ops.expert_rows, bf(5, 16), order)
    refuses("type", ops.expert_rows, bf(4, 16).double(), order)
    refuses("rows", ops.expert_rows, bf(16, 4).t(), order)
    refuses("int32", ops.expert_rows, bf(4, 16), order._replace(rows=i32(4, 2).long()))
    refuses("offsets", ops.expert_rows, bf(4, 16), order._replace(offsets=i32(1)))
    refuses("1 to 32", ops.expert_rows, bf(4, 16), order._replace(rows=i32(4, 33)))
    w = torch.zeros(4, 2)
    refuses("8, one for every slot", ops.combine_experts, bf(7, 16), w, order)
    refuses("w must", ops.combine_experts, bf(8, 16), w.double(), order)
    refuses("w must", ops.combine_experts, bf(8, 16), w[:, :1], order)
    refuses("CUDA", ops.combine_experts, bf(8, 16), w, order)
    refuses("CUDA", ops.expert_rows_backward, bf(8, 16), order)
    refuses("type", ops.combine_experts_backward, bf(4, 16), bf(8, 16).half(), w, order)
    refuses("rows of 24", ops.combine_experts_backward, bf(4, 16), bf(8, 24), w, order)
    refuses("CUDA", ops.combine_experts_backward, bf(4, 16), bf(8, 16), w, order)
    kept = ops.Checkpoint(torch.zeros(8, 40).to(torch.float8_e4m3fn), torch.zeros(8, 2, dtype=torch.uint8))
    refuses("CUDA", ops.combine_experts_backward, bf(4, 40), kept, w, order)
    refuses("scales", ops.combine_experts_backward, bf(4, 40), kept._replace(scales=kept.scales[:, :1]), w, order)
    refuses("codes", ops.combine_experts_backward, bf(4, 40), kept._replace(codes=bf(8, 40)), w, order)

    x, weight, off = bf(6, 24), bf(3, 16, 24), i32(4)
    refuses("CUDA", ops.expert_linear, x, weight, off)
    refuses("type", ops.expert_linear, x.float(), weight.float(), off)
    refuses("weight has type", ops.expert_linear, x, weight.half(), off)
    refuses("E = 2", ops.expert_linear, x, weight, i32(3))
    refuses("offsets", ops.expert_linear, x, weight, off.long())
    refuses("multiples of 8", ops.expert_linear, bf(6, 20), bf(3, 16, 20), off)
    refuses("multiples of 8", ops.expert_linear, x, bf(3, 12, 24), off)
    refuses("rows of 16", ops.expert_linear, bf(6, 16), weight, off)
    refuses("16 bytes", ops.expert_linear, bf(6, 25)[:, :24], weight, off)
    refuses("16 bytes", ops.expert_linear, x, bf(3, 16, 25)[:, :, :24], off)
    refuses("16 bytes", ops.expert_linear, x, bf(3, 24, 16).transpose(1, 2), off)
    dy = bf(6, 16)
    refuses("CUDA", ops.expert_linear_backward, dy, x, weight, off)
    refuses("rows of 24", ops.expert_linear_backward, bf(6, 24), x, weight, off)
    refuses("x must be", ops.expert_linear_backward, dy, bf(5, 24), weight, off)
    refuses("x is needed", ops.expert_linear_backward, dy, None, weight, off)
    refuses("add must", ops.expert_linear_backward, dy, x, weight, off, add=bf(6, 16))
    refuses("16 bytes", ops.expert_linear_backward, dy, x, weight, off, add=bf(6, 25)[:, :24])
    refuses("not asked for", ops.expert_linear_backward, dy, x, weight, off, add=x, need_dx=False)
    refuses("dw_dtype", ops.expert_linear_backward, dy, x, weight, off, dw_dtype=torch.float16)

    refuses("CUDA", ops.checkpoint, x)
    refuses("type", ops.checkpoint, x.double())
    refuses("CUDA", ops.restore, kept, torch.bfloat16)
    refuses("dtype", ops.restore, kept, torch.float64)
    refuses("dtype", ops.restore, kept, None)
    refuses("codes", ops.restore, kept._replace(codes=kept.codes.t()), torch.bfloat16)
    refuses("CUDA", ops.gated, x, x)
    refuses("type", ops.gated, x.float(), x.float())
    refuses("up must", ops.gated, x, x[:5])
    refuses("act", ops.gated, x, x, act="tanh")
    refuses("CUDA", ops.gated_backward, x, x, x)
    refuses("gate must", ops.gated_backward, x, x[:5], x)
    refuses("both", ops.gated_backward, bf(8, 40), kept, bf(8, 40))
    refuses("must be", ops.gated_backward, bf(7, 40), kept, kept)

    refuses("CUDA", ops.linear_backward, bf(8, 16), kept, bf(16, 40), need_dw=False)
    refuses("dy must", ops.linear_backward, dy, kept, bf(16, 40))
    odd = ops.Checkpoint(torch.zeros(8, 12).to(torch.float8_e4m3fn), torch.zeros(8, 1, dtype=torch.uint8))
    refuses("multiple of 8", ops.linear_backward, bf(8, 16), odd, bf(16, 16)[:, :12])
    refuses("z must", ops.linear_backward, dy, x, bf(16, 24), z=kept, act="silu")
    refuses("z is needed", ops.linear_backward, dy, x, bf(16, 24), z=kept)
    refuses("keep", Experts, weight, weight, bf(3, 24, 16), keep="4 bits")
    refuses("expected", Experts, weight, weight, bf(3, 16, 24))


def test_the_references_gradients_against_differences():
    """Central differences of the float64 references, exact for what is linear in each argument."""
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    ids = torch.tensor([[0, 2], [2, 2], [1, -1], [7, 0]], dtype=torch.int32)
    slots, rows, offsets = X.order(ids, 3)
    assert offsets.tolist() == [0, 2, 3, 6] and slots.tolist() == [0, 7, 4, 1, 2, 3, -1, -1]
    assert rows.tolist() == [[0, 3], [4, 5], [2, -1], [-1, 1]]
    r, w, dy = rnd(8, 5), rnd(4, 2), rnd(4, 5)
    dr, dw, _ = X.combine_backward(dy, r, w, rows, 8)
    f = lambda r, w: (X.combine(r, w, rows)[0] * dy).sum()  # noqa: E731
    for t, d, at in ((r, dr, (3, 1)), (r, dr, (7, 0)), (w, dw, (1, 1)), (w, dw, (2, 1))):
        e = torch.zeros_like(t)
        e[at] = 0.5
        diff = f(r + e, w) - f(r - e, w) if t is r else f(r, w + e) - f(r, w - e)
        assert abs(diff - d[at]) < 1e-12
    x, weight, d = rnd(8, 4), rnd(3, 4, 6), rnd(8, 6)
    dw, _ = X.weights_grad(d, x, offsets)
    dx, _ = X.products(d, weight.transpose(1, 2), offsets)
    f = lambda x, weight: (X.products(x, weight, offsets)[0] * d).sum()  # noqa: E731
    for i, j in ((0, 1), (5, 3), (6, 2)):
        e = torch.zeros_like(x)
        e[i, j] = 0.5
        assert abs(f(x + e, weight) - f(x - e, weight) - dx[i, j]) < 1e-12
    e = torch.zeros_like(weight)
    e[2, 1, 5] = 0.5
    assert abs(f(x, weight + e) - f(x, weight - e) - dw[2, 5, 1]) < 1e-12


def test_the_reference_encoding():
    x = torch.tensor([[448.0, 17.0, 19.0, -0.3], [449.0, 17.0, 1.0, 2.0 ** -9]])
    code, unit = X.encode(x)
    assert unit.tolist() == [[1.0], [2.0]]
    assert code[0].tolist() == [448.0, 16.0, 20.0, -0.3125]  # ties to even
    assert (X.decode(code, unit) - x.double()).abs().max() <= 2.0 ** -4 * 449
    assert R.U32 == 2.0 ** -24
