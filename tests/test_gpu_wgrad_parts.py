"""Weight gradients whose rows are split into parts, to the bit: dy and x are
small whole numbers, so that every product and every partial sum is a whole
number below 2^24 (at most 20000 rows of 3 * 8, and 1000 to add to: 481000), which
fp32 holds whatever the order, and a row lost, doubled or of a neighbour shows."""
import ctypes

import pytest
import torch

import moe_expert_load_ue_amd as ue
from gpu_helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
M = 20000


def parts_of(ctx, N, K, groups):
    p = ue.ue_weight_grad_product(M=M, N=N, K=K, groups=groups)
    return ue.library().ue_weight_grad_workspace(ctx._h, ctypes.byref(p)) // (groups * N * K * 4)


# parts of a group of n rows are n / parts rows, rounded up past the next multiple of
# 64: lengths around 64 * parts, around one part and below it, no rows, and all rows
ONE = [[5, 5 + n] for n in (0, 1, 63, 64, 65, 127, 128, 129, 4095, 4096, 4097, 8191, 8192, 8193,
                            M - 5)]
SEVERAL = [[0, 1, 1, 9000, M], [3, 4098, 4098, 8195, 8260], [0, 64, 127, 4224, 4224],
           [0, M, M, M, M], [0, 0, 0, 0, M], [7, 2054, 4102, 6151, 19999]]


@pytest.mark.parametrize("N,K,parts,offs", [(70, 90, 64, ONE), (128, 128, 64, ONE), (300, 520, 34, ONE),
                                            (96, 160, 19, SEVERAL), (128, 64, 19, SEVERAL)])
@pytest.mark.parametrize("packed", [False, True])
def test_split_sums_are_exact(N, K, parts, offs, packed):
    ctx = ue.Context(8, 1, 0, 2, 64, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(N + K)
    whole = lambda top, *s: torch.randint(-top, top + 1, s, generator=g, device=DEV)  # noqa: E731
    dy, x = whole(3, M, N), whole(8, M, K)
    base = whole(1000, len(offs[0]) - 1, N, K).float()
    index = torch.randint(-9, M + 9, (M,), generator=g, device=DEV).int()
    there = (index >= 0) & (index < M)
    dyt, xt, xs = dy.bfloat16(), x.bfloat16(), None
    if packed:
        xt, xs = ue.ue_pack_rows(ctx, xt)
        assert torch.equal(ue.ue_unpack_rows(ctx, xt, xs).long(), x)
    groups = len(offs[0]) - 1
    assert parts_of(ctx, N, K, groups) == parts
    for at in (None, index):
        rows = x if at is None else torch.where(there[:, None], x[index.clamp(0, M - 1).long()], 0)
        for off in offs:
            say("split sums", N, K, packed, at is not None, off)
            want = torch.zeros((groups, N, K), device=DEV)
            for i in range(groups):
                r = slice(off[i], off[i + 1])
                want[i] = torch.matmul(dy[r].double().t().contiguous(), rows[r].double()).float()
            o = torch.tensor(off, dtype=torch.int32, device=DEV)
            out = torch.full((groups, N, K), float("nan"), device=DEV)
            ue.ue_weight_grad(ctx, dyt, xt, xs, o, at, out=out)
            assert torch.equal(out, want)
            out = base.clone()
            ue.ue_weight_grad(ctx, dyt, xt, xs, o, at, out=out, accumulate=True)
            assert torch.equal(out, want + base)
    ctx.close()


@pytest.mark.parametrize("packed", [False, True])
def test_sums_without_a_workspace_are_exact(packed):
    """The same through the library without a workspace: not split."""
    say("unsplit sums", packed)
    ctx = ue.Context(8, 1, 0, 2, 64, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    N, K = 72, 96
    dy = torch.randint(-3, 4, (M, N), generator=g, device=DEV)
    x = torch.randint(-8, 9, (M, K), generator=g, device=DEV)
    dyt, xt, xs = dy.bfloat16(), x.bfloat16(), None
    if packed:
        xt, xs = ue.ue_pack_rows(ctx, xt)
    out = torch.full((N, K), float("nan"), device=DEV)
    p = ue.ue_weight_grad_product(
        dy=dyt.data_ptr(), x=xt.data_ptr(), x_scale=xs.data_ptr() if packed else None,
        out=out.data_ptr(), lddy=N, ldx=K, lds=K // 32, ldo=K, out_stride=N * K, x_rows=M, groups=1,
        index_div=1, M=M, N=N, K=K)
    stream = torch.cuda.current_stream().cuda_stream
    assert ue.library().ue_weight_grad(ctx._h, ctypes.byref(p), stream) == 0
    assert torch.equal(out, torch.matmul(dy.double().t().contiguous(), x.double()).float())
    ctx.close()
