"""Packed rows of the largest finite numbers stand for finite numbers, and what
is made of them is finite where the values are."""
import numpy as np
import pytest
import torch

import moe_expert_load_ue_amd as ue
from gpu_helpers import say
from oracle import train as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
EDGE = np.float32(127 * 2.0 ** 121)
# the border and its neighbours, the largest numbers of fp32 and of bf16
TOPS = np.array([np.finfo(np.float32).max, np.float32(255 * 2.0 ** 120), EDGE,
                 np.nextafter(EDGE, np.float32(0)), np.nextafter(EDGE, np.float32(np.inf)),
                 np.float32(3.2e38), np.float32(2.0 ** 127)], np.float32)


def rows():
    x = np.zeros((2 * TOPS.size, 64), np.float32)
    x[::2, 3], x[1::2, 40] = TOPS, -TOPS
    x[:, 7], x[:, 50], x[:, 9] = 2.0 ** 120, -3 * 2.0 ** 121, 1.0
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_pack_and_unpack(dtype):
    say("pack the largest", dtype)
    ctx = ue.Context(8, 1, 0, 2, 8, device=DEV)
    x = torch.from_numpy(rows()).to(dtype)
    x = x[torch.isfinite(x).all(1)]              # (bf16 rounds some to infinity)
    assert x.shape[0] >= 6
    q, s = ue.ue_pack_rows(ctx, x.to(DEV))
    wq, ws = R.pack(x.double().numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)
    for t in (torch.float32, torch.bfloat16):
        v = ue.ue_unpack_rows(ctx, q, s, out_dtype=t)
        assert bool(torch.isfinite(v).all())
        assert np.array_equal(v.double().cpu().numpy(), R.unpack(wq, ws))
    ctx.close()


def test_gated_gradient():
    """gate = +-top: s is 1 or 0, so dgate = dh up s and dup = dh gate s, finite
    for small dh; h overflows or is 0 as the values do."""
    say("gated gradient of the largest")
    ctx = ue.Context(8, 1, 0, 2, 8, device=DEV)
    x = rows()
    gu = np.concatenate([x, np.full_like(x, 0.5)], 1)
    h, q, s = ue.ue_gated(ctx, torch.from_numpy(gu).to(DEV))
    dh = np.full(x.shape, 2.0 ** -60, np.float32)
    dgu, again = ue.ue_gated_backward(ctx, torch.from_numpy(dh).to(DEV), q, s)
    gate, up = R.kept(gu)
    want, wh = R.gated_backward(gate, up, dh)
    got = dgu.double().cpu().numpy()
    # products of four factors with s within 8 u, 1 + gate (1 - s) exactly 1 or
    # with s = 0: 26 u of the values, as for any other
    assert np.all(np.abs(got - want) <= 26 * U * np.abs(want) + 1e-36)
    assert np.all(np.abs(again.double().cpu().numpy() - wh) <= 12 * U * np.abs(wh) + 1e-36)
    ctx.close()


def test_weight_gradient_of_a_row_without_gradient():
    """A row of dy that is zero adds nothing, whatever the tokens are."""
    say("weight gradient beside the largest")
    ctx = ue.Context(8, 1, 0, 2, 8, device=DEV)
    x = torch.from_numpy(rows()).to(DEV)
    q, s = ue.ue_pack_rows(ctx, x)
    dy = torch.zeros((x.shape[0], 24), device=DEV).bfloat16()
    assert not bool((ue.ue_weight_grad(ctx, dy, q, s) != 0).any())
    dy[3, 5] = 2.0 ** -100
    got = ue.ue_weight_grad(ctx, dy, q, s)[0]
    want = torch.from_numpy(R.unpack(q.cpu().numpy(), s.cpu().numpy())).to(DEV)[3] * 2.0 ** -100
    assert torch.equal(got[5].double(), want)
    got[5] = 0
    assert not bool((got != 0).any())
    ctx.close()
