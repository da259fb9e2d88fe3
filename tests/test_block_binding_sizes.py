"""Sizes that do not fit the C entry points' int32 are refused by the binding: cut to their lower half
they would name another, valid size.  No GPU needed (the sizes are looked at before the tensors)."""
import os

import pytest
import torch

from mxfp4_mixture_experts_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.library_path()), reason="library not built")

WRAPPED = [(1 << 32) + 4, -(1 << 32) + 4, 1 << 31, -(1 << 31) - 1]


@pytest.mark.parametrize("v", WRAPPED)
def test_workspace_queries(v):
    for call in (lambda: B.moe_norm_backward_workspace_size(v, 64), lambda: B.moe_norm_backward_workspace_size(4, v),
                 lambda: B.moe_combine_norm_backward_workspace_size(v, 64),
                 lambda: B.moe_combine_norm_backward_workspace_size(4, v),
                 lambda: B.moe_balance_workspace_size(v, 32, 1), lambda: B.moe_balance_workspace_size(4, v, 1),
                 lambda: B.moe_balance_workspace_size(4, 32, v)):
        with pytest.raises(B.MXFP4Error, match="int32") as e:
            call()
        assert e.value.status == 1


@pytest.mark.parametrize("v", WRAPPED)
def test_calls(v):
    h, f, i = torch.zeros(64, dtype=torch.bfloat16), torch.zeros(64), torch.zeros(64, dtype=torch.int32)
    for call in (lambda: B.moe_norm(h, h, v, 8, h), lambda: B.moe_norm(h, h, 4, v, h),
                 lambda: B.moe_norm_backward(h, h, h, v, 8, h), lambda: B.moe_norm_backward(h, h, h, 4, v, h),
                 lambda: B.moe_combine_norm(f, None, v, 1, 8, h, h), lambda: B.moe_combine_norm(f, None, 4, v, 8, h, h),
                 lambda: B.moe_combine_norm(f, None, 4, 1, v, h, h),
                 lambda: B.moe_combine_norm_backward(h, f, f, v, 1, 8), lambda: B.moe_combine_norm_backward(h, f, f, 4, v, 8),
                 lambda: B.moe_combine_norm_backward(h, f, f, 4, 1, v),
                 lambda: B.moe_balance(h, i, v, 8, 1, i, i, f), lambda: B.moe_balance(h, i, 4, v, 1, i, i, f),
                 lambda: B.moe_balance(h, i, 4, 8, v, i, i, f), lambda: B.moe_balance(h, i, 4, 8, 1, i, i, f, i, v),
                 lambda: B.moe_route_backward(h, i, f, f, v, 8, 1, f), lambda: B.moe_route_backward(h, i, f, f, 4, v, 1, f),
                 lambda: B.moe_route_backward(h, i, f, f, 4, 8, v, f),
                 lambda: B.moe_route_backward(h, i, f, f, 4, 8, 1, f, i, v, i, i, f)):
        with pytest.raises(B.MXFP4Error, match="int32"):
            call()


def test_sizes_in_range_pass_on():
    assert B.moe_norm_backward_workspace_size(4, 64) == 4 * 64 * 4
    with pytest.raises(B.MXFP4Error, match="workspace query"):
        B.moe_norm_backward_workspace_size(-(1 << 31), 64)
    with pytest.raises(ValueError, match="device tensor"):
        B.moe_norm(torch.zeros(8, dtype=torch.bfloat16), None, 1, 8, torch.zeros(8, dtype=torch.bfloat16))
