"""What ue_combine_backward_all refuses, on the CPU: what ue_combine_backward
does, and to do without dy."""
import moe_expert_load_ue_amd as ue
from test_train_refusals import A, EINVAL, ESHAPE, ODD, T, check, ctx  # noqa: F401


def test_refusals(ctx):  # noqa: F811
    good = dict(dout=A, type=1, lddout=40, inv_perm=A, weights=A, y=A, ldy=40, rows=7, T=4, H=40,
                dy=A, lddy=40, dweights=A, workspace=None, stream=None)
    check(ctx, "ue_combine_backward_all", good, [
        (EINVAL, dict(dy=None)), (EINVAL, dict(dy=None, T=0)), (EINVAL, dict(dout=None)),
        (EINVAL, dict(type=2)), (ESHAPE, dict(lddout=39)), (EINVAL, dict(inv_perm=None)),
        (EINVAL, dict(weights=ODD)), (EINVAL, dict(y=None)), (ESHAPE, dict(ldy=39)),
        (ESHAPE, dict(rows=-1)), (ESHAPE, dict(T=T + 1)), (ESHAPE, dict(T=-1)), (ESHAPE, dict(H=0)),
        (ESHAPE, dict(H=(1 << 20) + 1)), (ESHAPE, dict(lddy=39)), (EINVAL, dict(dy=ODD)),
        (EINVAL, dict(dweights=A + 2)), (EINVAL, dict(workspace=A + 8)),
        # rows that are found with notes need room for these
        (EINVAL, dict(rows=(1 << 20) + 1))])
    f = ue.library().ue_combine_backward_workspace
    assert f(None, 1, 1) == f(ctx, -1, 1) == f(ctx, 1, -1) == 0
    assert f(ctx, 1 << 14, 1 << 20) == 0 and f(ctx, 0, 1 << 20) == 0
    assert f(ctx, (1 << 14) + 1, 5) == 20 and f(ctx, 0, (1 << 20) + 1) == 4 * ((1 << 20) + 1)
