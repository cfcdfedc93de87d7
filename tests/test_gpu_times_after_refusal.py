"""A call of the training step that is refused leaves the kernel times of the call
before."""
import ctypes

import pytest
import torch

import moe_expert_load_ue_amd as ue
from gpu_helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_weight_grad_of_too_many_tiles():
    say("kernel times after a refusal")
    ctx = ue.Context(32, 1, 0, 2, 3000, device=DEV)
    x = torch.randn((3000, 32), device=DEV)
    ue.ue_set_timing(ctx, True)
    ue.ue_balance(ctx, x, x.topk(2, 1).indices.int())
    before = ue.ue_kernel_times(ctx)
    assert len(before) == 2
    some = torch.zeros(64, device=DEV).data_ptr()     # (that nothing reads)
    # more tiles than a launch holds: refused on the host
    p = ue.ue_weight_grad_product(
        dy=some, x=some, offsets=some, out=some, lddy=1 << 20, ldx=1000, ldo=1000,
        out_stride=1000 << 20, x_rows=8, groups=(1 << 20) - 1, index_div=1, M=8, N=1 << 20, K=1000)
    stream = torch.cuda.current_stream().cuda_stream
    assert ue.library().ue_weight_grad(ctx._h, ctypes.byref(p), stream) == -2
    assert ue.ue_kernel_times(ctx) == before
    ctx.close()
