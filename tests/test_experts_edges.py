"""Refusals at the edges of the operators on expert rows, in C and on torch tensors; no GPU."""
import ctypes

import pytest
import torch

from tests.test_experts_refusals import ROWS
from tile_signaled_grouped_gb300 import capi, ops


@pytest.mark.parametrize("T,topk", [(1 << 60, 16), (1 << 62, 4), (1 << 62, 32), ((1 << 30) + 1, 1), ((1 << 25) + 1, 32)])
def test_rows_refuse_more_tokens_than_any_product_tells(T, topk):
    """T * topk above 2^30, also where the product of 64 bits is 0 or negative."""
    lib = capi.lib()
    for f in (lib.moe_expert_rows, lib.moe_combine_experts, lib.moe_combine_experts_backward):
        a = capi.moe_rows_args(**{**ROWS, "T": T, "topk": topk})
        assert f(ctypes.byref(a), None) == capi.MOE_ERR_ARG


def test_a_gradient_without_weights_is_refused_by_name():
    """combine_experts takes no weights; its backward pass, which has none to give a gradient of, says what to call."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    order = ops.ExpertOrder(*(torch.zeros(*s, dtype=torch.int32) for s in ((8,), (4, 2), (9,))))
    with pytest.raises(ValueError, match="expert_rows"):
        ops.combine_experts_backward(bf(4, 16), bf(8, 16), None, order)
