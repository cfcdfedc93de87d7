"""The gradient of the experts' rows that ue_combine_backward makes itself is
whole: rows that no assignment names are zeros, whatever lay in the memory
before; rows of a caller's own dy stay as they are."""
import numpy as np
import pytest
import torch

import moe_expert_load_ue_amd as ue
from gpu_helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")


def spoil(rows, H, dtype):
    """Leaves NaN in the memory that the next tensors of this size get."""
    full = [torch.full((rows, H), NAN, dtype=dtype, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    del full


def wanted(dout, inv, w, rows):
    """Row by row from the definition: zeros, then w dout where named (products
    of two fp32 numbers, or of a bf16 and an fp32 one, rounded once each way)."""
    dy = torch.zeros((rows, dout.shape[1]), dtype=dout.dtype, device=DEV)
    named = (inv >= 0) & (inv < rows)
    t, j = named.nonzero(as_tuple=True)
    dy[inv[t, j].long()] = (dout[t].float() * w[t, j][:, None]).to(dout.dtype)
    return dy


def assigned(g, T, k, rows, lost):
    """Places of T x k assignments, distinct, some outside the rows."""
    inv = torch.randperm(max(rows, T * k) + 3, generator=g, device=DEV)[:T * k].int()
    gone = torch.rand(T * k, generator=g, device=DEV) < lost
    return torch.where(gone, -1 - inv % 5, inv).view(T, k)


@pytest.mark.parametrize("T,k,H,rows,lost", [
    (1, 1, 1, 1, 1.0), (1, 8, 700, 8, 0.3), (5, 3, 33, 40, 0.0), (9, 2, 3, 18, 0.5), (130, 6, 96, 780, 0.1),
    (200, 4, 1000, 3000, 0.0), (513, 2, 130, 511, 0.0), (700, 8, 257, 5600, 0.02),
    # rows of many workgroups' shares, none named, all named
    (4096, 8, 64, 32768, 0.25), (9, 1, 520, 140001, 0.0), (3000, 2, 40, 6000, 1.0),
    (3000, 2, 40, 6000, 0.0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_without_an_assignment_are_zeros(T, k, H, rows, lost, dtype):
    say("combine, all rows", T, k, H, rows, lost, dtype)
    ctx = ue.Context(max(k, 8), 1, 0, k, T, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(T + H)
    inv = assigned(g, T, k, rows, lost)
    if lost == 0.0 and rows == T * k:
        inv = torch.randperm(rows, generator=g, device=DEV).int().view(T, k)
    dout = torch.randn((T, H), generator=g, device=DEV).to(dtype)
    y = torch.randn((rows, H), generator=g, device=DEV).to(dtype)
    w = torch.rand((T, k), generator=g, device=DEV)
    want = wanted(dout, inv, w, rows)
    for _ in range(2):
        spoil(rows, H, dtype)
        dy, dw = ue.ue_combine_backward(ctx, dout, inv, w, y)
        assert torch.equal(dy, want)
    own = torch.full((rows, H), -7.0, dtype=dtype, device=DEV)
    _, dw2 = ue.ue_combine_backward(ctx, dout, inv, w, y, dy=own)
    named = torch.zeros(rows + 1, dtype=torch.bool, device=DEV)
    named[torch.where((inv >= 0) & (inv < rows), inv, rows).view(-1).long()] = True
    assert torch.equal(own[named[:rows]], want[named[:rows]])
    assert bool((own[~named[:rows]] == -7).all()) and torch.equal(dw, dw2)
    # without y the gradient has a row for every assignment
    want = wanted(dout, inv, w, T * k)
    spoil(T * k, H, dtype)
    dy, none = ue.ue_combine_backward(ctx, dout, inv, w)
    assert none is None and torch.equal(dy, want)
    # a stream of its own
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dy2, _ = ue.ue_combine_backward(ctx, dout, inv, w, stream=side)
    side.synchronize()
    assert torch.equal(dy2, want)
    ctx.close()


def test_no_tokens_leave_zeros():
    say("combine, all rows, no tokens")
    ctx = ue.Context(8, 1, 0, 2, 8, device=DEV)
    none = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    for H in (1, 5, 130, 1000):
        y = torch.ones((50, H), device=DEV)
        spoil(50, H, torch.float32)
        dy, dw = ue.ue_combine_backward(ctx, torch.empty((0, H), device=DEV), none, y=y)
        assert dy.shape == (50, H) and not bool((dy != 0).any()) and dw.shape == (0, 2)
    dy, _ = ue.ue_combine_backward(ctx, torch.empty((0, 7), device=DEV), none,
                                   y=torch.empty((0, 7), device=DEV))
    assert dy.shape == (0, 7)
    ctx.close()


@pytest.mark.parametrize("T,k,rows", [(1 << 13, 4, 1 << 15), ((1 << 13) + 1, 4, 1 << 15),
                                      (1 << 13, 4, 1 << 20), (1 << 13, 4, (1 << 20) + 1),
                                      (1 << 18, 4, 1 << 20), (1 << 19, 4, 1 << 21), (100, 4, 3 << 20),
                                      ((1 << 25) + 3, 1, (1 << 25) + 9)])
def test_many_rows(T, k, rows):
    """On both sides of the sizes where all assignments are looked at and where
    rows are found with notes, and more than one launch of assignments."""
    say("combine, many rows", T, k, rows)
    ctx = ue.Context(8, 1, 0, k, T, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(rows)
    for H in (3, 130) if T < 1 << 25 else (1,):
        inv = assigned(g, T, k, rows, 0.1)
        dout = torch.randn((T, H), generator=g, device=DEV).bfloat16()
        y = torch.randn((rows, H), generator=g, device=DEV).bfloat16()
        w = torch.rand((T, k), generator=g, device=DEV)
        want = wanted(dout, inv, w, rows)
        spoil(rows, H, torch.bfloat16)
        dy, _ = ue.ue_combine_backward(ctx, dout, inv, w, y)
        assert torch.equal(dy, want)
    ctx.close()


@pytest.mark.parametrize("junk", [0, 1, 5, 0x7FFFFFFF, -1])
def test_whatever_the_workspace_holds(junk):
    """Notes of rows that nobody names hold what was there: any number, one of an
    assignment among them, names nothing by itself."""
    say("combine, all rows, workspace", junk)
    T, k, H, rows = 9000, 4, 12, 40000
    ctx = ue.Context(8, 1, 0, k, T, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    inv = assigned(g, T, k, rows, 0.3)
    inv[0, :2] = torch.tensor([-1, -1], dtype=torch.int32)
    inv[1, 1] = rows + 7
    dout = torch.randn((T, H), generator=g, device=DEV)
    w = torch.rand((T, k), generator=g, device=DEV)
    dy = torch.full((rows, H), NAN, device=DEV)
    lib = ue.library()
    assert lib.ue_combine_backward_workspace(ctx._h, T, rows) == 4 * rows
    ws = torch.full((rows + 4,), junk, dtype=torch.int32, device=DEV)
    for _ in range(2):                       # the second time with its own notes
        rc = lib.ue_combine_backward_all(
            ctx._h, dout.data_ptr(), 0, H, inv.data_ptr(), w.data_ptr(), None, 0, rows, T, H,
            dy.data_ptr(), H, None, ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        assert torch.equal(dy, wanted(dout, inv, w, rows))
        assert bool((ws[rows:] == junk).all())
        inv = inv.flip(0).contiguous()       # other rows by the same assignments
        inv[5:900] = -1
    ctx.close()


@pytest.mark.parametrize("T", [300, 9000])
def test_graph_replays(T):
    """Captured with lost assignments, replayed with others between."""
    say("combine, all rows, graph", T)
    k, H = 4, 72
    ctx = ue.Context(8, 1, 0, k, T, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(9)
    dout = torch.randn((T, H), generator=g, device=DEV)
    w = torch.rand((T, k), generator=g, device=DEV)
    inv = assigned(g, T, k, T * k, 0.2)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ue.ue_combine_backward(ctx, dout, inv, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dy, _ = ue.ue_combine_backward(ctx, dout, inv, w)
    for n in range(4):
        say("replay", n)
        inv.copy_(assigned(g, T, k, T * k, 0.2 * n))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dy, wanted(dout, inv, w, T * k))
        assert torch.equal(dy, ue.ue_combine_backward(ctx, dout, inv, w)[0])
    ctx.close()


def test_rows_apart_through_the_library():
    """The library's call on rows apart: all rows written, nothing between."""
    say("combine, all rows, apart")
    T, k, H, rows = 40, 3, 37, 150
    ctx = ue.Context(8, 1, 0, k, T, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    inv = assigned(g, T, k, rows, 0.2)
    dout = torch.randn((T, H), generator=g, device=DEV)
    w = torch.rand((T, k), generator=g, device=DEV)
    wide = torch.full((rows, H + 11), -7.0, device=DEV)
    rc = ue.library().ue_combine_backward_all(
        ctx._h, dout.data_ptr(), 0, H, inv.data_ptr(), w.data_ptr(), None, 0, rows, T, H,
        wide.data_ptr(), H + 11, None, None, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(wide[:, :H], wanted(dout, inv, w, rows))
    assert bool((wide[:, H:] == -7).all())
    # more rows, none of them named
    rows = 1 << 21
    ws = torch.zeros(rows, dtype=torch.int32, device=DEV)
    wide = torch.full((rows, 5), -7.0, device=DEV)
    inv = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    rc = ue.library().ue_combine_backward_all(
        ctx._h, dout.data_ptr(), 0, H, inv.data_ptr(), w.data_ptr(), None, 0, rows, T, 3,
        wide.data_ptr(), 5, None, ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert not bool((wide[:, :3] != 0).any()) and bool((wide[:, 3:] == -7).all())
    ctx.close()
