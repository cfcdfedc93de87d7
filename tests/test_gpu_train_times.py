"""Kernel times of the training step's calls: one for each kernel that a call
launches."""
import pytest
import torch

import moe_expert_load_ue_amd as ue
from gpu_helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_a_time_for_each_kernel():
    say("kernel times of the training step")
    ctx = ue.Context(32, 1, 0, 2, 3000, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((3000, 32), generator=g, device=DEV)
    ids = x.topk(2, 1).indices.int()
    dy = torch.randn((20000, 96), generator=g, device=DEV).bfloat16()
    v = torch.randn((20000, 160), generator=g, device=DEV).bfloat16()
    inv = torch.randperm(6000, generator=g, device=DEV).int().view(3000, 2)
    y = torch.randn((6000, 40), generator=g, device=DEV)
    ue.ue_set_timing(ctx, True)

    def times(call):
        out = call()
        t = ue.ue_kernel_times(ctx)
        assert all(n > 0 for n in t)
        return out, len(t)
    assert ue.ue_balance_workspace(ctx, 3000) > 0 == ue.ue_balance_workspace(ctx, 100)
    (_, counts, _), n = times(lambda: ue.ue_balance(ctx, x, ids))
    assert n == 2                            # shares, and their sum
    assert times(lambda: ue.ue_balance(ctx, x[:100], ids[:100]))[1] == 1
    one = torch.ones(1, device=DEV)
    assert times(lambda: ue.ue_balance_backward(ctx, x, counts, one))[1] == 1
    (q, s), n = times(lambda: ue.ue_pack_rows(ctx, x))
    assert n == 1 and times(lambda: ue.ue_unpack_rows(ctx, q, s))[1] == 1
    (h, gq, gs), n = times(lambda: ue.ue_gated(ctx, x))
    assert n == 1 and times(lambda: ue.ue_gated_backward(ctx, h, gq, gs))[1] == 1
    assert times(lambda: ue.ue_combine(ctx, y, inv))[1] == 1
    assert times(lambda: ue.ue_combine_backward(ctx, y[:3000], inv, y=y))[1] == 1
    # many assignments: notes of who names a row, then the gradient
    far = torch.randperm(40000, generator=g, device=DEV).int().view(20000, 2)
    big = ue.Context(32, 1, 0, 2, 20000, device=DEV)
    ue.ue_set_timing(big, True)
    ue.ue_combine_backward(big, dy.float(), far)
    assert len(ue.ue_kernel_times(big)) == 2
    big.close()
    # parts of a long sum, and their sum; a short one is one kernel
    assert times(lambda: ue.ue_weight_grad(ctx, dy, v))[1] == 2
    assert times(lambda: ue.ue_weight_grad(ctx, dy[:200], v[:200]))[1] == 1
    ctx.close()
