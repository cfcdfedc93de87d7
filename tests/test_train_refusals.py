"""What the training step's entry points refuse, through the C ABI on the CPU:
a refusal comes before any launch, so a context that has only its sizes will do
(made by a host-only shim from the library's own header), with addresses that
nothing reads."""
import ctypes
import os
import subprocess

import pytest

import moe_expert_load_ue_amd as ue
from moe_expert_load_ue_amd import build as B

SHIM = """
#include "ue_internal.h"
extern "C" void *make_ctx(int E, int k, int tokens) {
    ue_ctx *c = new ue_ctx;
    c->cfg.num_experts = c->E = E;
    c->cfg.topk = c->k = k;
    c->cfg.max_tokens = tokens;
    c->num_cu = 256;
    return c;
}
"""
E, K, T = 8, 2, 1024
BIG = 600                                # tokens that need a workspace
A, ODD = 1 << 20, (1 << 20) + 1          # an address, and one aligned to nothing
EINVAL, ESHAPE = -1, -2


@pytest.fixture(scope="module")
def ctx(tmp_path_factory):
    folder = str(tmp_path_factory.mktemp("shim"))
    src, lib = os.path.join(folder, "shim.hip"), os.path.join(folder, "shim.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run([B.hipcc(), "--offload-arch=gfx950", "--cuda-host-only", "-std=c++17",
                    "-shared", "-fPIC", "-I", B.CSRC, "-o", lib, src], check=True)
    make = ctypes.CDLL(lib).make_ctx
    make.restype = ctypes.c_void_p
    return make(E, K, T)


def check(ctx, name, good, bad):
    """`good`: arguments by name, in the call's order; `bad`: (status, changes)."""
    f = getattr(ue.library(), name)
    for code, change in bad:
        assert set(change) <= set(good), change
        args = list({**good, **change}.values())
        assert f(ctx, *args) == code, (name, change)
        assert ue.library().ue_last_error(ctx).decode().startswith(name), change
    assert f(None, *good.values()) == EINVAL


def test_balance(ctx):
    good = dict(logits=A, type=0, ld=E, T=4, score=0, ids=A, offsets=A, n_seq=3, counts=A,
                prob=A, loss=A, workspace=A, stream=None)
    check(ctx, "ue_balance", good, [
        (EINVAL, dict(logits=None)), (EINVAL, dict(type=2)), (ESHAPE, dict(ld=E - 1)),
        (ESHAPE, dict(T=-1)), (ESHAPE, dict(T=T + 1)), (EINVAL, dict(score=2)),
        (EINVAL, dict(ids=None)), (ESHAPE, dict(n_seq=-1)), (ESHAPE, dict(n_seq=(1 << 20) + 1)),
        (ESHAPE, dict(offsets=None)), (ESHAPE, dict(offsets=None, n_seq=0)),
        (EINVAL, dict(counts=None)), (EINVAL, dict(prob=None)), (EINVAL, dict(loss=None)),
        (EINVAL, dict(workspace=None, T=BIG)), (EINVAL, dict(workspace=A + 8)),
        (EINVAL, dict(logits=A + 2)), (EINVAL, dict(logits=ODD, type=1)),
        (EINVAL, dict(ids=A + 2)), (EINVAL, dict(offsets=ODD)), (EINVAL, dict(counts=ODD)),
        (EINVAL, dict(prob=ODD)), (EINVAL, dict(loss=ODD))])
    lib = ue.library()
    assert lib.ue_balance_workspace(ctx, -1, 1) == 0 == lib.ue_balance_workspace(None, 1, 1)
    # shares of 64 tokens and a slot for every share and sequence, 8 bytes an
    # expert; none for few tokens
    assert lib.ue_balance_workspace(ctx, BIG, 5) == (10 + 5) * E * 8
    assert lib.ue_balance_workspace(ctx, 512, 5) == 0


def test_balance_backward(ctx):
    good = dict(logits=A, type=1, ld=E, T=4, score=1, offsets=A, n_seq=3, counts=A, dloss=A,
                dlogits=A, ld_out=E, accumulate=0, stream=None)
    check(ctx, "ue_balance_backward", good, [
        (EINVAL, dict(logits=None)), (EINVAL, dict(type=-1)), (ESHAPE, dict(ld=E - 1)),
        (ESHAPE, dict(ld_out=E - 1)), (ESHAPE, dict(T=T + 1)), (EINVAL, dict(score=-1)),
        (ESHAPE, dict(offsets=None)), (EINVAL, dict(counts=None)), (EINVAL, dict(dloss=None)),
        (EINVAL, dict(dlogits=None)), (EINVAL, dict(dlogits=ODD)), (EINVAL, dict(counts=ODD)),
        (EINVAL, dict(dloss=A + 2))])


def test_pack_and_unpack(ctx):
    good = dict(x=A, type=0, ldx=40, M=3, K=40, q=A, ldq=64, scale=A, lds=2, stream=None)
    bad = [(EINVAL, dict(x=None)), (EINVAL, dict(type=2)), (ESHAPE, dict(ldx=39)),
           (ESHAPE, dict(M=-1)), (ESHAPE, dict(K=0)), (ESHAPE, dict(K=(1 << 20) + 1)),
           (EINVAL, dict(q=None)), (EINVAL, dict(q=A + 8)), (ESHAPE, dict(ldq=48)),
           (ESHAPE, dict(ldq=72)), (EINVAL, dict(scale=None)), (ESHAPE, dict(lds=1)),
           (EINVAL, dict(x=A + 2))]
    check(ctx, "ue_pack_rows", good, bad)
    order = ("q", "ldq", "scale", "lds", "M", "K", "x", "type", "ldx", "stream")
    check(ctx, "ue_unpack_rows", {n: good[n] for n in order}, bad)


def test_gated(ctx):
    good = dict(gu=A, type=0, ldgu=80, M=3, I=40, h=A, ldh=40, q=A, ldq=128, scale=A, lds=4,
                stream=None)
    check(ctx, "ue_gated", good, [
        (EINVAL, dict(gu=None)), (EINVAL, dict(type=2)), (ESHAPE, dict(ldgu=79)),
        (ESHAPE, dict(M=-1)), (ESHAPE, dict(I=0)), (ESHAPE, dict(I=(1 << 19) + 1)),
        (EINVAL, dict(h=None)), (ESHAPE, dict(ldh=39)), (EINVAL, dict(q=None)),
        (EINVAL, dict(scale=None)), (ESHAPE, dict(ldq=112)), (ESHAPE, dict(ldq=136)),
        (ESHAPE, dict(lds=3)), (EINVAL, dict(q=A + 4)), (EINVAL, dict(gu=A + 2)),
        (EINVAL, dict(h=A + 1))])
    good = dict(q=A, ldq=128, scale=A, lds=4, dh=A, type=1, lddh=40, M=3, I=40, dgu=A, lddgu=80,
                h=A, ldh=40, stream=None)
    check(ctx, "ue_gated_backward", good, [
        (EINVAL, dict(q=None)), (EINVAL, dict(scale=None)), (ESHAPE, dict(ldq=112)),
        (ESHAPE, dict(lds=3)), (EINVAL, dict(dh=None)), (EINVAL, dict(type=3)),
        (ESHAPE, dict(lddh=39)), (ESHAPE, dict(M=-1)), (ESHAPE, dict(I=0)),
        (EINVAL, dict(dgu=None)), (ESHAPE, dict(lddgu=79)), (ESHAPE, dict(ldh=39)),
        (EINVAL, dict(h=ODD)), (EINVAL, dict(dgu=ODD))])


def test_weight_grad(ctx):
    lib = ue.library()
    base = dict(dy=A, x=A, x_scale=A, offsets=A, index=A, out=A, workspace=None, lddy=24, ldx=48,
                lds=2, ldo=40, out_stride=24 * 40, x_rows=5, groups=3, index_div=2, M=10, N=24,
                K=40, accumulate=0)

    def call(**kw):
        p = ue.ue_weight_grad_product(**{**base, **kw})
        return lib.ue_weight_grad(ctx, ctypes.byref(p), None)
    assert lib.ue_weight_grad(ctx, None, None) == EINVAL
    assert lib.ue_weight_grad(None, None, None) == EINVAL
    for kw in (dict(M=-1), dict(M=(1 << 30) + 1, x_rows=1 << 30), dict(N=-1), dict(K=-1), dict(N=(1 << 20) + 1), dict(K=(1 << 20) + 1),
               dict(x_rows=-1), dict(x_rows=0), dict(groups=-1), dict(groups=1 << 20),
               dict(offsets=None), dict(lddy=23), dict(ldx=40), dict(ldx=56), dict(lds=1),
               dict(ldo=39), dict(out_stride=24 * 40 - 1), dict(index_div=0), dict(index=None),
               dict(lddy=(1 << 24) + 1), dict(ldx=(1 << 24) + 16), dict(ldo=1 << 30),
               dict(x_scale=None, ldx=39)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(dy=None), dict(x=None), dict(out=None), dict(dy=ODD), dict(x=A + 8),
               dict(x=ODD, x_scale=None), dict(out=A + 2), dict(offsets=ODD), dict(index=A + 2),
               dict(workspace=A + 8)):
        assert call(**kw) == EINVAL, kw
    # nothing to write: no launch, and no pointer is needed
    for kw in (dict(N=0), dict(K=0), dict(groups=0)):
        assert call(dy=None, x=None, out=None, **kw) == 0, kw
    assert lib.ue_weight_grad_workspace(ctx, None) == 0


def test_combine(ctx):
    good = dict(y=A, type=0, ldy=40, rows=7, inv_perm=A, weights=A, add=A, ldadd=40, T=4, H=40,
                out=A, ldo=40, stream=None)
    check(ctx, "ue_combine", good, [
        (EINVAL, dict(y=None)), (EINVAL, dict(type=2)), (ESHAPE, dict(ldy=39)),
        (ESHAPE, dict(rows=-1)), (EINVAL, dict(inv_perm=None)), (EINVAL, dict(inv_perm=A + 2)),
        (EINVAL, dict(weights=A + 2)), (ESHAPE, dict(ldadd=39)), (EINVAL, dict(add=A + 2)),
        (ESHAPE, dict(T=-1)), (ESHAPE, dict(T=T + 1)), (ESHAPE, dict(H=0)),
        (ESHAPE, dict(H=(1 << 20) + 1)), (EINVAL, dict(out=None)), (ESHAPE, dict(ldo=39)),
        (EINVAL, dict(out=ODD))])
    good = dict(dout=A, type=1, lddout=40, inv_perm=A, weights=A, y=A, ldy=40, rows=7, T=4, H=40,
                dy=A, lddy=40, dweights=A, stream=None)
    check(ctx, "ue_combine_backward", good, [
        (EINVAL, dict(dout=None)), (EINVAL, dict(type=2)), (ESHAPE, dict(lddout=39)),
        (EINVAL, dict(inv_perm=None)), (EINVAL, dict(weights=ODD)), (EINVAL, dict(y=None)),
        (ESHAPE, dict(ldy=39)), (ESHAPE, dict(rows=-1)), (ESHAPE, dict(T=T + 1)),
        (ESHAPE, dict(H=0)), (ESHAPE, dict(lddy=39)), (EINVAL, dict(dy=ODD)),
        (EINVAL, dict(dweights=A + 2))])
