"""The training step's operators on the GPU against their 64-bit definitions
(oracle/train.py).

Tolerances, u = 2^-24 and u16 = 2^-8 (half a step of fp32 and of bf16):
- scores: an exponential within 4 u, its sigmoid within 8 u; a softmax argument
  is rounded, which the exponential shows |argument| u of (arguments here below
  32); a sum over up to 1024 experts adds at most 16 + 6 roundings: p within
  8 + 32 + 4 + 22 + 2 = 68 u.
- prob: positive terms; a lane adds at most (share / 4) of them, a share 20
  lanes' and waves' sums, a sequence its shares in 16 runs: at most 64 + 20 + 32
  more for the sizes here: 200 u; loss: E more in a tree and two factors: 230 u.
- dlogits: p, then p c and their dot within 68 + 26 u of the terms' magnitudes,
  the sigmoid's slope 8 u, three factors: 120 u of p (c + sum p c) f, twice that
  for the difference of two such; bf16 adds u16 of the value.
- packed rows: equal to the bit.
- gated: silu within 9 u, with up 10 u. Backward: s and 1 - s within 8 u each;
  s (1 + gate (1 - s)) within 8 u + 12 u |gate| (1 - s) <= 0.28 (its largest
  value for negative gates, where terms cancel) s: at most 24 u of s (1 + |gate|
  (1 - s)); times dh up 2 u more. Exponentials below 2^-126 are 0.
- weight gradients: n terms in some order: (n + 2) u of the sum of their
  magnitudes, whichever way the matrix units round, twice.
- combine: k + 1 additions and as many products fused: (k + 2) u of the terms'
  magnitudes; dots over H in lanes' runs of H / 64 / 4 and a tree: (H / 64 + 20) u.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_ue_amd as ue
from gpu_helpers import say
from oracle import train as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")
U, U16 = 2.0 ** -24, 2.0 ** -8
F32, BF16 = torch.float32, torch.bfloat16
TYPES = [F32, BF16]


def ctx_for(E=8, k=2, T=64):
    return ue.Context(E, 1, 0, k, T, device=DEV)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def rounded(a, dtype):
    """a as `dtype` holds it, in float64."""
    return torch.from_numpy(np.asarray(a)).to(dtype).double().numpy()


def half_step(dtype, want):
    return (U16 if dtype == BF16 else U) * np.abs(want)


def close(got, want, tol):
    got, tol = np.asarray(got), np.broadcast_to(tol, np.shape(want))
    bad = ~((np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want)) | (got == want))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           got[bad][:4], want[bad][:4], tol[bad][:4])


def as_held(want):
    """Infinite where the value is past the largest float (and its half step)."""
    return np.where(np.abs(want) >= 2.0 ** 128 * (1 - 2.0 ** -25), np.sign(want) * INF, want)


def pitched(a, dtype, gap, fill=-7.0):
    """a on the device as rows `gap` elements further apart than wide."""
    t = torch.full((a.shape[0], a.shape[1] + gap), fill, dtype=dtype, device=DEV)
    t[:, :a.shape[1]] = dev(a, dtype)
    return t[:, :a.shape[1]]


# ---- balance loss -------------------------------------------------------------

def balance_case(rng, T, E, k, dtype, masked):
    x = rounded(rng.normal(size=(T, E)) * 2, dtype)
    if masked:
        x[rng.random((T, E)) < 0.4] = -INF
        x[::5] = -INF
    ids = np.argsort(-x, 1, kind="stable")[:, :k].astype(np.int32)
    ids[np.isneginf(np.take_along_axis(x, ids.astype(np.int64), 1))] = -1
    return x, ids


def check_balance(ctx, x, ids, off, dtype, score, gap=0, **kw):
    T, E = x.shape
    k = ids.shape[1]
    rng = np.random.default_rng(T + E)
    lg = pitched(x, dtype, gap) if gap else dev(x, dtype)
    o = None if off is None else dev(np.asarray(off, np.int32))
    loss, counts, prob = ue.ue_balance(ctx, lg, dev(ids), o, score, **kw)
    wl, wc, wp = R.balance(x, ids, off, score)
    assert np.array_equal(host(counts), wc)
    close(host(prob), wp, 200 * U * wp)
    close(host(loss), wl, 230 * U * wl)
    dloss = rng.normal(size=len(wl)).astype(np.float32)
    d = ue.ue_balance_backward(ctx, lg, counts, dev(dloss), o, score, **kw)
    want, size = R.balance_backward(x, wc, dloss, k, off, score)
    assert d.dtype == dtype
    close(host(d), want, 240 * U * size + half_step(dtype, want) + 1e-37)
    # added to what is there, in fp32; rows of no sequence stay
    base = rounded(rng.normal(size=(T, E)) * np.abs(want).max(), dtype)
    acc = dev(base, dtype)
    ue.ue_balance_backward(ctx, lg, counts, dev(dloss), o, score, dlogits=acc,
                           accumulate=True, **kw)
    close(host(acc), base + want,
          240 * U * size + half_step(dtype, base + want) + half_step(F32, base + want) + 1e-37)


BALANCE = [(1, 1, 1), (5, 8, 2), (63, 32, 3), (64, 33, 4), (65, 60, 6), (130, 64, 8),
           (77, 100, 7), (200, 128, 8), (90, 130, 8), (257, 256, 8), (31, 300, 3),
           (40, 512, 16), (9, 1000, 5), (6, 1024, 100)]


@pytest.mark.parametrize("T,E,k", BALANCE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
def test_balance(T, E, k, score, dtype):
    rng = np.random.default_rng(T * 1000 + E)
    ctx = ctx_for(E, k, T)
    for masked in (False, True):
        x, ids = balance_case(rng, T, E, k, dtype, masked)
        cuts = np.sort(rng.integers(0, T + 1, size=4))
        for off in (None, [0, T], [int(v) for v in cuts], [0, 0, T // 2, T // 2, T]):
            say("balance", T, E, k, score, dtype, masked, off)
            check_balance(ctx, x, ids, off, dtype, score)
    ctx.close()


def test_balance_many_and_clamped_sequences():
    """More sequences than tokens, one token each, offsets outside the tokens,
    shares that hold many sequences and sequences of many shares."""
    rng = np.random.default_rng(1)
    T, E, k = 700, 24, 3
    ctx = ctx_for(E, k, T)
    x, ids = balance_case(rng, T, E, k, F32, False)
    for off in (list(range(T + 1)), [-5, 3, 3, T + 9], [T, T + 1], [0] * 40 + [T] * 40,
                [0, 1, 2, 3, 690], sorted(rng.integers(0, T, size=1500).tolist()), [5]):
        say("balance sequences", len(off), off[:4])
        check_balance(ctx, x, ids, off, F32, "softmax")
    ctx.close()


def test_balance_among_empty_sequences():
    """A million empty sequences in one place, and offsets that decrease: each
    workgroup looks past them, none goes round in circles."""
    say("balance among empty sequences")
    T, E, k = 1000, 32, 2
    ctx = ctx_for(E, k, T)
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((T, E), generator=g, device=DEV)
    ids = x.topk(k, 1).indices.int()
    n = 1 << 20
    off = torch.full((n + 1,), 333, dtype=torch.int32, device=DEV)
    off[0], off[-2:] = 0, torch.tensor([700, 1000], dtype=torch.int32)
    loss, counts, prob = ue.ue_balance(ctx, x, ids, off)
    few = torch.tensor([0, 333, 700, 1000], dtype=torch.int32, device=DEV)
    want = ue.ue_balance(ctx, x, ids, few)
    keep = torch.tensor([0, n - 2, n - 1], device=DEV)
    assert torch.equal(loss[keep], want[0]) and torch.equal(counts[keep], want[1])
    assert torch.equal(prob[keep], want[2])
    assert int((loss != 0).sum()) == 3 and int(counts.sum()) == T * k
    d = ue.ue_balance_backward(ctx, x, counts, torch.ones(n, device=DEV), off)
    assert torch.equal(d, ue.ue_balance_backward(ctx, x, want[1], torch.ones(3, device=DEV), few))
    for bad in ([1000, 500, 0], [0, 900, 100, 1000, 50, 600], [-7, 2000, -7, 2000]):
        bad = torch.tensor(bad, dtype=torch.int32, device=DEV)
        loss, counts, _ = ue.ue_balance(ctx, x, ids, bad)
        ue.ue_balance_backward(ctx, x, counts, loss, bad)
    torch.cuda.synchronize()
    ctx.close()


@pytest.mark.parametrize("E", [24, 30])
@pytest.mark.parametrize("dtype", TYPES)
def test_balance_strides(E, dtype):
    rng = np.random.default_rng(E)
    T, k = 150, 4
    ctx = ctx_for(E, k, T)
    x, ids = balance_case(rng, T, E, k, dtype, True)
    for gap in (1, 4, 8):
        say("balance strides", E, dtype, gap)
        check_balance(ctx, x, ids, [3, 70, 149], dtype, "sigmoid", gap)
    # the gradient over the logits themselves, and into rows apart
    lg = dev(x, dtype)
    _, counts, _ = ue.ue_balance(ctx, lg, dev(ids))
    one = torch.ones(1, device=DEV)
    want = ue.ue_balance_backward(ctx, lg, counts, one)
    apart = pitched(np.zeros((T, E)), dtype, 3)
    ue.ue_balance_backward(ctx, lg, counts, one, dlogits=apart)
    # (rows whose alignment differs may share a token's experts out to other
    # lanes, so its sums may be in another order: each within its tolerance)
    exact, size = R.balance_backward(x, host(counts), [1], k, None, "softmax")
    for got in (apart, want):
        close(host(got), exact, 240 * U * size + half_step(dtype, exact) + 1e-37)
    assert bool((torch.as_strided(apart, (T, 3), (E + 3, 1), E) == -7).all())
    assert ue.ue_balance_backward(ctx, lg, counts, one, dlogits=lg) is lg
    assert torch.equal(lg, want)
    ctx.close()


@pytest.mark.parametrize("E", [2, 3, 5, 30, 131, 442, 777])
@pytest.mark.parametrize("n", [1, 9, 62, 63, 64, 65, 300])
def test_balance_in_shares(E, n):
    """Batches that many workgroups share, of few and of many sequences, with
    experts that are no multiple of four and padding ahead and behind."""
    say("balance in shares", E, n)
    rng = np.random.default_rng(E * 1000 + n)
    T, k = 1237, 2
    ctx = ctx_for(E, k, T)
    assert ue.ue_balance_workspace(ctx, T, n) > 0
    x, ids = balance_case(rng, T, E, k, F32, False)
    off = np.sort(rng.integers(0, T + 1, size=n + 1))
    check_balance(ctx, x, ids, off, F32, "sigmoid" if n % 2 else "softmax")
    ctx.close()


def test_balance_special_values():
    """NaN spoils its sequence's loss and prob and its own token's gradient
    only; +inf is the largest float; ids outside the experts are not counted."""
    E, k = 6, 2
    ctx = ctx_for(E, k, 8)
    low = float(np.finfo(np.float32).min)
    x = np.array([[0, 1, 2, 3, 4, 5], [1, np.nan, 0, 0, 0, 0], [INF, 0, INF, 0, -INF, 1],
                  [low] * 6, [-INF] * 6, [-INF] * 5 + [2]], np.float32)
    ids = np.array([[5, 4], [0, 7], [0, 2], [-1, 1], [-1, -1], [5, -9]], np.int32)
    off = [0, 1, 2, 6]
    for score in ("softmax", "sigmoid"):
        loss, counts, prob = ue.ue_balance(ctx, dev(x), dev(ids), dev(np.array(off, np.int32)),
                                           score)
        wl, wc, wp = R.balance(x, ids, off, score)
        assert np.array_equal(host(counts), wc)
        assert np.isnan(host(loss)[1]) and np.isnan(host(prob)[1]).all()
        for s in (0, 2):
            close(host(prob)[s], wp[s], 200 * U * wp[s])
            close(host(loss)[s], wl[s], 230 * U * wl[s])
        d = host(ue.ue_balance_backward(ctx, dev(x), counts, torch.ones(3, device=DEV),
                                        dev(np.array(off, np.int32)), score))
        keep = [0, 2, 3, 4, 5]
        want, size = R.balance_backward(np.delete(x, 1, 0), wc[[0, 2]], [1, 1], k, [0, 1, 5], score)
        close(d[keep], want, 240 * U * size + 1e-30)
        assert np.isnan(d[1]).all() and np.all(d[4] == 0)
    ctx.close()


def test_balance_of_nothing():
    ctx = ctx_for(8, 2, 8)
    empty = torch.empty((0, 8), device=DEV)
    ids = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    loss, counts, prob = ue.ue_balance(ctx, empty, ids)
    assert host(loss).tolist() == [0] and not host(counts).any() and not host(prob).any()
    off = torch.zeros(1, dtype=torch.int32, device=DEV)       # no sequence at all
    x = torch.randn((3, 8), device=DEV)
    loss, counts, prob = ue.ue_balance(ctx, x, torch.zeros((3, 2), dtype=torch.int32, device=DEV), off)
    assert loss.numel() == 0 and counts.shape == (0, 8)
    d = ue.ue_balance_backward(ctx, x, counts, loss, off)
    assert not host(d).any()
    assert ue.ue_balance_backward(ctx, empty, counts, loss, off).shape == (0, 8)
    ctx.close()


def test_balance_of_a_large_batch_repeats():
    """Counts and sums over many shares, against float64 on the device; the same
    bits on a second call."""
    T, E, k = 70001, 256, 8
    ctx = ctx_for(E, k, T)
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((T, E), generator=g, device=DEV)
    ids = x.topk(k, 1).indices.int()
    off = torch.tensor([0, 11, 30000, 30000, 70000], dtype=torch.int32, device=DEV)
    loss, counts, prob = ue.ue_balance(ctx, x, ids, off)
    again = ue.ue_balance(ctx, x, ids, off)
    for a, b in zip(again, (loss, counts, prob)):
        assert torch.equal(a, b)
    dl = torch.rand(4, generator=g, device=DEV)
    d = ue.ue_balance_backward(ctx, x, counts, dl, off)
    p = torch.softmax(x.double(), 1)
    for s, (a, b) in enumerate(((0, 11), (11, 30000), (30000, 30000), (30000, 70000))):
        n = max(b - a, 1)
        c = torch.bincount(ids[a:b].reshape(-1).long(), minlength=E).double()
        assert torch.equal(counts[s].long(), c.long())
        mean = p[a:b].sum(0) / n
        assert bool(((prob[s].double() - mean).abs() <= 300 * U * mean).all())
        want = E / (k * n) * (c * mean).sum()
        assert abs(float(loss[s]) - float(want)) <= 330 * U * float(want)
        f = float(dl[s]) * E / (k * n * n)
        dot = (p[a:b] * c).sum(1, keepdim=True)
        want = f * p[a:b] * (c - dot)
        tol = 240 * U * abs(f) * p[a:b] * (c + dot) + 1e-37
        assert bool(((d[a:b].double() - want).abs() <= tol).all())
    assert not bool(d[70000:].any())
    ctx.close()


# ---- packed rows ----------------------------------------------------------------

def pack_case(rng, M, K, dtype):
    x = rng.normal(size=(M, K)) * np.exp2(rng.integers(-130, 120, size=(M, 1)))
    x[rng.random((M, K)) < 0.05] = 0
    x[M // 2, :] = 0
    x[:, 0] *= np.exp2(rng.integers(-3, 8, size=M))
    return rounded(np.clip(x, -3e38, 3e38), dtype)


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (2, 31), (5, 32), (4, 33), (7, 100), (64, 256),
                                 (9, 1000), (3, 2049)])
@pytest.mark.parametrize("dtype", TYPES)
def test_pack_rows(M, K, dtype):
    rng = np.random.default_rng(M * 100 + K)
    ctx = ctx_for()
    x = pack_case(rng, M, K, dtype)
    wq, ws = R.pack(x)
    for gap in (0, 1, 8):
        say("pack", M, K, dtype, gap)
        q, s = ue.ue_pack_rows(ctx, pitched(x, dtype, gap))
        assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)
        pad = -K % 32
        if pad:
            P = K + pad
            assert not torch.as_strided(q, (M, pad), (P, 1), K).any()
        for t in TYPES:
            v = ue.ue_unpack_rows(ctx, q, s, out_dtype=t)
            assert v.dtype == t and np.array_equal(host(v), R.unpack(wq, ws))
        out = pitched(np.zeros((M, K)), dtype, gap + 3)
        ue.ue_unpack_rows(ctx, q, s, out=out)
        assert np.array_equal(host(out), R.unpack(wq, ws))
    # into rows given by the caller, apart, what lies between left alone
    P = (K + 31) // 32 * 32
    q = torch.full((M, P + 16), -9, dtype=torch.int8, device=DEV)
    s = torch.full((M, P // 32 + 5), 9, dtype=torch.uint8, device=DEV)
    ue.ue_pack_rows(ctx, dev(x, dtype), q=q[:, :K], scale=s[:, :P // 32])
    assert np.array_equal(host(q)[:, :K], wq) and np.array_equal(host(s)[:, :P // 32], ws)
    assert (host(q)[:, P:] == -9).all() and (host(s)[:, P // 32:] == 9).all()
    ctx.close()


def test_pack_special_values():
    """Every magnitude of bf16 as a block's largest, ties, infinities, NaN and
    the smallest numbers."""
    ctx = ctx_for()
    tops = np.arange(1, 0x7F80, dtype=np.uint32)[:, None] << 16
    x = np.zeros((tops.shape[0], 32), np.float32)
    x[:, 5:6] = tops.view(np.float32)
    x[:, 6:7] = -(tops.view(np.float32) / np.float32(2))
    x[:, 7:8] = (tops & 0xFFC00000).view(np.float32)
    wq, ws = R.pack(x)
    for dtype in TYPES:
        xt = torch.from_numpy(x).to(dtype)
        if dtype == BF16:
            wq, ws = R.pack(xt.double().numpy())
        q, s = ue.ue_pack_rows(ctx, xt.to(DEV))
        assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)
    x = np.zeros((4, 96), np.float32)
    x[0, 33], x[1, 1], x[2, 95] = INF, np.nan, -INF
    x[:, 34] = 3.0
    x[3, :] = np.float32(1e-45)
    q, s = ue.ue_pack_rows(ctx, dev(x))
    wq, ws = R.pack(x)
    assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)
    close(host(ue.ue_unpack_rows(ctx, q, s)), R.unpack(wq, ws), 0)
    assert ue.ue_pack_rows(ctx, torch.empty((0, 40), device=DEV))[1].shape == (0, 2)
    ctx.close()


# ---- gated activation -------------------------------------------------------------

def check_gated(h, gu, dtype):
    gu = np.asarray(gu)
    want = R.gated(gu)
    # silu is 0 where exp(-v) is past the largest float, v < -88.72: there it is
    # below 88.73 e^-88.72 = 2.7e-37 in magnitude
    lost = 3e-37 * (1 + np.abs(gu[:, gu.shape[1] // 2:]))
    close(host(h), as_held(want), 10 * U * np.abs(want) + half_step(dtype, want) + lost)


def check_gated_backward(dgu, h, gate, up, dh, dtype):
    want, wh = R.gated_backward(gate, up, dh)
    s = R._sigmoid(gate)
    rest = R._sigmoid(-gate)
    size = np.concatenate([np.abs(dh * up) * s * (1 + np.abs(gate) * rest),
                           np.abs(dh * gate) * s], 1)
    close(host(dgu), as_held(want), 26 * U * size + half_step(dtype, want) + 1e-36 * (1 + np.abs(
        np.concatenate([dh * up, dh], 1))))
    if h is not None:
        close(host(h), as_held(wh), 12 * U * np.abs(wh) + half_step(dtype, wh) + 1e-36 * (1 + np.abs(up)))


@pytest.mark.parametrize("M,I", [(1, 1), (3, 5), (2, 32), (5, 33), (7, 40), (33, 96), (9, 501),
                                 (64, 256), (3, 1030)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gated(M, I, dtype):
    rng = np.random.default_rng(M * 7 + I)
    ctx = ctx_for()
    gu = rounded(rng.normal(size=(M, 2 * I)) * np.exp(rng.normal(size=(M, 1))) * 3, dtype)
    dh = rounded(rng.normal(size=(M, I)), dtype)
    P = (I + 31) // 32 * 32
    for gap in (0, 1, 8):
        say("gated", M, I, dtype, gap)
        h, q, s = ue.ue_gated(ctx, pitched(gu, dtype, gap))
        check_gated(h, gu, dtype)
        assert q.shape == (M, 2 * P) and s.shape == (M, P // 16)
        for half, a in ((gu[:, :I], 0), (gu[:, I:], P)):
            wq, ws = R.pack(half)
            assert np.array_equal(host(q)[:, a:a + I], wq)
            assert not host(q)[:, a + I:a + P].any()
            assert np.array_equal(host(s)[:, a // 32:(a + P) // 32], ws)
            # each half is packed rows of its own
            v = ue.ue_unpack_rows(ctx, q[:, a:a + I], s[:, a // 32:(a + P) // 32])
            assert np.array_equal(host(v), R.unpack(wq, ws))
        gate, up = R.kept(gu)
        dgu, again = ue.ue_gated_backward(ctx, pitched(dh, dtype, gap), q, s)
        check_gated_backward(dgu, again, gate, up, dh, dtype)
        only, none = ue.ue_gated_backward(ctx, dev(dh, dtype), q, s, with_h=False)
        assert none is None and torch.equal(only, dgu)
        out, oh = pitched(np.zeros((M, 2 * I)), dtype, gap + 2), pitched(np.zeros((M, I)), dtype, gap)
        ue.ue_gated_backward(ctx, dev(dh, dtype), q, s, dgu=out, h=oh)
        assert torch.equal(out, dgu) and torch.equal(oh, again)
        bare, nq, ns = ue.ue_gated(ctx, dev(gu, dtype), keep=False)
        assert nq is None and ns is None and torch.equal(bare, h)
    ctx.close()


def test_gated_extremes():
    """Gates over the whole range, where exponentials overflow and underflow;
    a block with a NaN spoils itself only."""
    ctx = ctx_for()
    g = np.concatenate([np.linspace(-200, 200, 401), [-3e38, 3e38, 1e-30, -1e-30, 0.0, -0.0, -87.4,
                                                     -88.8, -103.9, 88.8, 30.0]])
    gu = np.zeros((g.size, 64), np.float32)
    gu[:, 0] = g
    gu[:, 32] = 1.5
    h, q, s = ue.ue_gated(ctx, dev(gu))
    check_gated(h, gu, F32)
    gate, up = R.kept(gu)
    dh = np.full((g.size, 32), -0.75, np.float32)
    dgu, again = ue.ue_gated_backward(ctx, dev(dh), q, s)
    check_gated_backward(dgu, again, gate, up, dh, F32)
    gu = np.ones((2, 128), np.float32)
    gu[0, 40], gu[1, 70] = np.nan, INF
    h, q, s = ue.ue_gated(ctx, dev(gu))
    d, _ = ue.ue_gated_backward(ctx, torch.ones((2, 64), device=DEV), q, s)
    d = host(d)
    assert np.isnan(d[0, 32:64]).all() and not np.isnan(d[0, :32]).any()
    assert np.isnan(d[1, :32]).all() and not np.isnan(d[1, 32:64]).any()
    assert ue.ue_gated(ctx, torch.empty((0, 8), device=DEV))[0].shape == (0, 4)
    ctx.close()


def test_gated_gradient_against_differences():
    """The gradient against central differences of the forward kernel, at kept
    values (which packing leaves as they are)."""
    rng = np.random.default_rng(5)
    ctx = ctx_for()
    M, I, step = 6, 32, 2.0 ** -5
    gu = R.unpack(*R.pack(rng.normal(size=(M, 2 * I)) * 2))
    dh = rng.normal(size=(M, I)).astype(np.float32)
    _, q, s = ue.ue_gated(ctx, dev(gu, F32))
    d = host(ue.ue_gated_backward(ctx, dev(dh), q, s)[0])
    for j in (0, 3, 31, 32, 50, 63):
        v = [gu.copy(), gu.copy()]
        v[0][:, j] += step
        v[1][:, j] -= step
        up, down = (host(ue.ue_gated(ctx, dev(w, F32), keep=False)[0])[:, j % I] for w in v)
        # third derivative of silu below 0.5: step^2 / 6 of it, |up| below 8
        assert np.all(np.abs((up - down) / (2 * step) * dh[:, j % I] - d[:, j]) <=
                      (step ** 2 / 12 * 8 + 1e-4) * np.abs(dh[:, j % I]))
    ctx.close()


# ---- weight gradients ---------------------------------------------------------------

def wgrad_case(rng, rows, M, N, K, packed):
    dy = rounded(rng.normal(size=(M, N)), BF16)
    x = rounded(rng.normal(size=(rows, K)) * np.exp(rng.normal(size=(rows, 1))), BF16)
    if not packed:
        return dy, x, dev(x, BF16), None
    q, s = R.pack(x)
    P = (K + 31) // 32 * 32
    qt = torch.zeros((rows, P), dtype=torch.int8, device=DEV)
    qt[:, :K] = dev(q)
    return dy, R.unpack(q, s), qt[:, :K], dev(s)


def check_wgrad(got, dy, x, off, index, div, base=None):
    want, size = R.weight_grad(dy, x, off, index, div)
    terms = max([b - a for a, b in R._sequences(off, dy.shape[0])], default=0) + 2
    if base is not None:
        want, size = want + base, size + np.abs(base)
    close(host(got), want, 2 * terms * U * size)


GROUPED = [(40, 40, 24, 32, None), (7, 50, 33, 70, [0, 50]), (1, 1, 1, 1, None),
           (90, 300, 64, 64, [0, 0, 3, 67, 67, 299]), (64, 200, 130, 258, [0, 65, 129, 200]),
           (33, 77, 7, 500, [5, 70]), (500, 700, 257, 96, [0, 1, 33, 97, 350, 699, 700]),
           (128, 1100, 300, 520, [0, 1100]), (20, 64, 512, 40, [0, 32, 64])]


@pytest.mark.parametrize("rows,M,N,K,off", GROUPED)
@pytest.mark.parametrize("packed", [False, True])
def test_weight_grad(rows, M, N, K, off, packed):
    rng = np.random.default_rng(M + N + K)
    ctx = ctx_for()
    dy, x, xt, xs = wgrad_case(rng, rows, M, N, K, packed)
    dyt = dev(dy, BF16)
    o = None if off is None else dev(np.array(off, np.int32))
    G = 1 if off is None else len(off) - 1
    for div in (None, 1, 3):
        say("wgrad", rows, M, N, K, off, packed, div)
        if div is None:
            if rows < M:
                continue
            index, it = None, None
        else:
            index = rng.integers(-1, rows * div + 2, size=M).astype(np.int32)
            it = dev(index)
        out = torch.full((G, N, K), -7.0, device=DEV)
        ue.ue_weight_grad(ctx, dyt, xt, xs, o, it, div or 1, out=out)
        check_wgrad(out, dy, x, off, index, div or 1)
        again = ue.ue_weight_grad(ctx, dyt, xt, xs, o, it, div or 1)
        assert torch.equal(again, out)
        base = rng.normal(size=(G, N, K)).astype(np.float32)
        acc = dev(base)
        ue.ue_weight_grad(ctx, dyt, xt, xs, o, it, div or 1, out=acc, accumulate=True)
        check_wgrad(acc, dy, x, off, index, div or 1, base)
    ctx.close()


@pytest.mark.parametrize("packed", [False, True])
def test_weight_grad_strides(packed):
    """Rows and matrices apart, unaligned, what lies between left alone; clamped
    offsets."""
    rng = np.random.default_rng(11)
    rows, M, N, K = 50, 90, 45, 67
    ctx = ctx_for()
    dy, x, xt, xs = wgrad_case(rng, rows, M, N, K, packed)
    index = rng.integers(0, rows, size=M).astype(np.int32)
    off = [-3, 20, 20, 70, 1000]
    for gap in (0, 1, 5, 16):
        say("wgrad strides", packed, gap)
        dyt = pitched(dy, BF16, gap)
        if packed:
            q = torch.full((rows, 96 + 16 * gap), 99, dtype=torch.int8, device=DEV)
            q[:, :K] = xt
            sc = torch.full((rows, 3 + gap), 99, dtype=torch.uint8, device=DEV)
            sc[:, :3] = xs
            a, b = q[:, :K], sc[:, :3]
        else:
            a, b = pitched(x, BF16, gap), None
        big = torch.full((4, N + 2, K + gap), -7.0, device=DEV)
        out = big[:, :N, :K]
        ue.ue_weight_grad(ctx, dyt, a, b, dev(np.array(off, np.int32)), dev(index), out=out)
        check_wgrad(out, dy, x, off, index, 1)
        assert bool((big[:, N:] == -7).all()) and bool((big[:, :, K:] == -7).all())
    # a slice of the rows' bytes that starts off 16-byte pieces
    flat = torch.zeros(M * N + 1, dtype=BF16, device=DEV)
    flat[1:] = dev(dy, BF16).reshape(-1)
    out = ue.ue_weight_grad(ctx, flat[1:].view(M, N), xt, xs, None, dev(index))
    check_wgrad(out, dy, x, None, index, 1)
    ctx.close()


@pytest.mark.parametrize("packed", [False, True])
def test_weight_grad_of_nothing_and_of_infinities(packed):
    ctx = ctx_for()
    rng = np.random.default_rng(12)
    dy, x, xt, xs = wgrad_case(rng, 40, 40, 24, 40, packed)
    empty = ue.ue_weight_grad(ctx, dev(dy, BF16)[:0], xt, xs,
                              torch.zeros(4, dtype=torch.int32, device=DEV),
                              torch.empty(0, dtype=torch.int32, device=DEV))
    assert empty.shape == (3, 24, 40) and not host(empty).any()
    keep = torch.full((2, 24, 40), 5.0, device=DEV)
    ue.ue_weight_grad(ctx, dev(dy, BF16), xt, xs, torch.tensor([7, 7, 7], dtype=torch.int32, device=DEV),
                      out=keep, accumulate=True)
    assert bool((keep == 5).all())
    assert ue.ue_weight_grad(ctx, dev(dy, BF16), xt, xs,
                             torch.zeros(1, dtype=torch.int32, device=DEV)).shape == (0, 24, 40)
    # infinities and NaN of one group's rows reach that group's results only:
    # the last row of a group lies behind the rows of a tile's end
    dy[9, 3], dy[10, 5], dy[33, 2] = INF, np.nan, INF
    off = [0, 10, 11, 33, 40]
    got = host(ue.ue_weight_grad(ctx, dev(dy, BF16), xt, xs, dev(np.array(off, np.int32))))
    with np.errstate(invalid="ignore"):
        want, size = R.weight_grad(dy, x, off)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = np.isfinite(want)
    assert np.array_equal(got[~ok & ~np.isnan(want)], want[~ok & ~np.isnan(want)])
    assert np.all(np.abs(got[ok] - want[ok]) <= 40 * U * size[ok])
    ctx.close()


WGRAD_LARGE = [(3000, 6000, 520, 776, 5), (900, 4100, 1030, 2060, 3), (4096, 8192, 200, 300, 1),
               (70, 30000, 70, 90, 2), (2000, 2500, 2048, 1024, 9)]


@pytest.mark.parametrize("rows,M,N,K,G", WGRAD_LARGE)
@pytest.mark.parametrize("packed", [False, True])
def test_weight_grad_large(rows, M, N, K, G, packed):
    """Many rows and tiles, against float64 products on the device."""
    say("wgrad large", rows, M, N, K, G, packed)
    ctx = ctx_for()
    g = torch.Generator(device=DEV).manual_seed(M)
    dy = torch.randn((M, N), generator=g, device=DEV).bfloat16()
    x = torch.randn((rows, K), generator=g, device=DEV).bfloat16()
    index = torch.randint(0, rows, (M,), generator=g, device=DEV, dtype=torch.int32)
    cut = torch.randint(0, M + 1, (G - 1,), generator=g, device=DEV).sort().values
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), M)]).int()
    xs = None
    if packed:
        x, xs = ue.ue_pack_rows(ctx, x)
        v = ue.ue_unpack_rows(ctx, x, xs).double()
    else:
        v = x.double()
    base = torch.randn((G, N, K), generator=g, device=DEV)
    for acc in (False, True):
        out = base.clone()
        ue.ue_weight_grad(ctx, dy, x, xs, off, index, out=out, accumulate=acc)
        o = off.tolist()
        for i in range(G):
            r = slice(o[i], o[i + 1])
            a, b = dy[r].double().t().contiguous(), v[index[r].long()]
            want, size = a @ b, a.abs() @ b.abs()
            if acc:
                want, size = want + base[i].double(), size + base[i].double().abs()
            tol = 2 * (o[i + 1] - o[i] + 2) * U * size
            assert bool(((out[i].double() - want).abs() <= tol).all()), (acc, i)
    ctx.close()


# ---- combine -----------------------------------------------------------------------

@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 700), (5, 3, 33), (9, 2, 512), (33, 8, 520),
                                   (20, 9, 1027), (7, 20, 64), (130, 6, 96), (3, 8, 4104)])
@pytest.mark.parametrize("dtype", TYPES)
def test_combine(T, k, H, dtype):
    rng = np.random.default_rng(T * 100 + H)
    ctx = ctx_for(max(k, 8), k, T)
    inv = rng.permutation(T * k + 3)[:T * k].astype(np.int32)
    inv[rng.random(T * k) < 0.15] = -1
    inv = inv.reshape(T, k)
    inv[T // 2] = -5                        # a token that found no place
    rows = T * k + 1                        # places past it count as none
    y = rounded(rng.normal(size=(rows, H)), dtype)
    w = rng.normal(size=(T, k)).astype(np.float32)
    add = rounded(rng.normal(size=(T, H)), dtype)
    dout = rounded(rng.normal(size=(T, H)), dtype)
    for gap, weights, ad in ((0, w, None), (1, None, add), (8, w, add)):
        say("combine", T, k, H, dtype, gap)
        wt = None if weights is None else dev(weights)
        at = None if ad is None else pitched(ad, dtype, gap)
        yt = pitched(y, dtype, gap)
        out = ue.ue_combine(ctx, yt, dev(inv), wt, add=at)
        want, size = R.combine(y, inv, weights, ad)
        assert out.dtype == dtype
        close(host(out), want, (k + 2) * U * size + half_step(dtype, want))
        into = pitched(np.zeros((T, H)), dtype, gap + 2)
        ue.ue_combine(ctx, yt, dev(inv), wt, add=at, out=into)
        assert torch.equal(into, out)
        dy = torch.full((rows, H), -7.0, dtype=dtype, device=DEV)
        dyt, dw = ue.ue_combine_backward(ctx, pitched(dout, dtype, gap), dev(inv), wt, yt, dy=dy)
        wy, wd, ws = R.combine_backward(dout, y, inv, weights)
        assert dyt is dy
        named = ~np.isnan(wy[:, 0])
        assert np.all(host(dy)[~named] == -7)
        close(host(dy)[named], wy[named], half_step(dtype, wy[named]) + 1e-40)
        close(host(dw), wd, (H / 64 + 20) * U * ws)
        # either gradient alone
        dy2 = torch.full((rows, H), -7.0, dtype=dtype, device=DEV)
        _, none = ue.ue_combine_backward(ctx, dev(dout, dtype), dev(inv), wt, dy=dy2)
        assert none is None and torch.equal(dy2, dy)
        no, dw2 = ue.ue_combine_backward(ctx, dev(dout, dtype), dev(inv), wt, yt, with_dy=False)
        assert no is None
        close(host(dw2), wd, (H / 64 + 20) * U * ws)
    # over what is added
    res = dev(add, dtype)
    assert ue.ue_combine(ctx, dev(y, dtype), dev(inv), dev(w), add=res, out=res) is res
    want, size = R.combine(y, inv, w, add)
    close(host(res), want, (k + 2) * U * size + half_step(dtype, want))
    ctx.close()


@pytest.mark.parametrize("H", (3, 5, 9, 17, 131, 257, 513, 515, 1027))
@pytest.mark.parametrize("dtype", TYPES)
def test_combine_rows_that_end_inside_a_piece(dtype, H):
    """Rows whose last piece reaches back into the one before: added to in place,
    with nothing written past their ends, infinities in that piece."""
    say("combine ends", H, dtype)
    T, k = 700, 2
    rng = np.random.default_rng(H)
    ctx = ctx_for(8, k, T)
    inv = rng.permutation(T * k).astype(np.int32).reshape(T, k)
    y = rounded(rng.normal(size=(T * k, H)), dtype)
    add = rounded(rng.normal(size=(T, H)), dtype)
    dout = rounded(1.0 + rng.random(size=(T, H)), dtype)
    w = rng.normal(size=(T, k)).astype(np.float32)
    wide = torch.full((T, H + 9), -7.0, dtype=dtype, device=DEV)
    res = wide[:, 4:4 + H]
    res.copy_(dev(add, dtype))
    assert ue.ue_combine(ctx, dev(y, dtype), dev(inv), dev(w), add=res, out=res) is res
    want, size = R.combine(y, inv, w, add)
    close(host(res), want, (k + 2) * U * size + half_step(dtype, want))
    assert bool((wide[:, :4] == -7).all()) and bool((wide[:, 4 + H:] == -7).all())
    y[5, H - 2] = INF
    wide = torch.full((T * k, H + 9), -7.0, dtype=dtype, device=DEV)
    dy, dw = ue.ue_combine_backward(ctx, dev(dout, dtype), dev(inv), dev(w), dev(y, dtype),
                                    dy=wide[:, 4:4 + H])
    wy, wd, ws = R.combine_backward(dout, y, inv, w)
    close(host(dy), wy, half_step(dtype, wy) + 1e-40)
    assert bool((wide[:, :4] == -7).all()) and bool((wide[:, 4 + H:] == -7).all())
    at = inv == 5
    got = host(dw)
    assert got[at] == INF
    close(got[~at], wd[~at], (H / 64 + 20) * U * ws[~at])
    ctx.close()


@pytest.mark.parametrize("shape", ((0,), (5,), (3, 7), (3, 0), (0, 4), (2, 3, 5), (2, 0, 5), (2, 3, 0)))
def test_outputs_made_here_are_ordinary_tensors(shape):
    """Their layout and device are torch.empty's, on the default stream and on
    another."""
    ctx = ctx_for(8, 2, 8)
    for stream in (None, torch.cuda.Stream()):
        for dtype in (torch.float32, torch.bfloat16, torch.int8, torch.int32):
            t = ue._new(shape, dtype, ctx, stream)
            w = torch.empty(shape, dtype=dtype, device=DEV)
            assert t.shape == w.shape and t.stride() == w.stride() and t.dtype == w.dtype
            assert t.device == w.device and t.is_contiguous() and not t.requires_grad
    ctx.close()


@pytest.mark.parametrize("H", (3, 100, 250, 2056))
@pytest.mark.parametrize("dtype", TYPES)
def test_large_sums_of_rows_are_the_small_ones(dtype, H):
    """A call that reads more than is kept in the caches, against two that read
    half of it: bit for bit."""
    say("large combine", H, dtype)
    k, es = 2, torch.finfo(dtype).bits // 8
    T = (140 << 20) // (H * es * k)
    ctx = ctx_for(8, k, T)
    g = torch.Generator(device=DEV).manual_seed(H)
    y = torch.randn((T * k, H), generator=g, device=DEV, dtype=dtype)
    dout = torch.randn((T, H), generator=g, device=DEV, dtype=dtype)
    w = torch.rand((T, k), generator=g, device=DEV)
    inv = torch.randperm(T * k, generator=g, device=DEV).int().view(T, k)
    out = ue.ue_combine(ctx, y, inv, w, add=dout)
    dy, dw = ue.ue_combine_backward(ctx, dout, inv, w, y)
    dy2 = torch.empty_like(dy)
    for part in (slice(0, T // 2), slice(T // 2, T)):
        assert torch.equal(out[part], ue.ue_combine(ctx, y, inv[part], w[part], add=dout[part]))
        _, dw2 = ue.ue_combine_backward(ctx, dout[part], inv[part], w[part], y, dy=dy2)
        assert torch.equal(dw[part], dw2)
    assert torch.equal(dy, dy2)
    ctx.close()


@pytest.mark.parametrize("I", (5, 302, 2048))
@pytest.mark.parametrize("dtype", TYPES)
def test_large_gated_rows_are_the_small_ones(dtype, I):
    """The same of the gated activation, its backward pass and packed rows."""
    say("large gated", I, dtype)
    es = torch.finfo(dtype).bits // 8
    M = (280 << 20) // (I * 2 * es)
    ctx = ctx_for(8, 2, 8)
    g = torch.Generator(device=DEV).manual_seed(I)
    gu = torch.randn((M, 2 * I), generator=g, device=DEV, dtype=dtype)
    dh = torch.randn((M, I), generator=g, device=DEV, dtype=dtype)
    h, q, s = ue.ue_gated(ctx, gu)
    dgu, h2 = ue.ue_gated_backward(ctx, dh, q, s)
    pq, ps = ue.ue_pack_rows(ctx, gu)
    bare = ue.ue_gated(ctx, gu, keep=False)[0]
    assert torch.equal(bare, h)
    for i in range(4):
        part = slice(M * i // 4, M * (i + 1) // 4)
        a = ue.ue_gated(ctx, gu[part])
        assert torch.equal(h[part], a[0]) and torch.equal(q[part], a[1]) and torch.equal(s[part], a[2])
        assert torch.equal(h[part], ue.ue_gated(ctx, gu[part], keep=False)[0])
        b = ue.ue_gated_backward(ctx, dh[part], q[part], s[part])
        assert torch.equal(dgu[part], b[0]) and torch.equal(h2[part], b[1])
        c = ue.ue_pack_rows(ctx, gu[part])
        assert torch.equal(pq[part], c[0]) and torch.equal(ps[part], c[1])
    ctx.close()


def test_combine_edges():
    """No tokens, no rows, infinities beside ordinary rows, the gather's
    gradient."""
    ctx = ctx_for(8, 2, 8)
    y = torch.randn((4, 16), device=DEV)
    none = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    assert ue.ue_combine(ctx, y, none).shape == (0, 16)
    assert ue.ue_combine_backward(ctx, torch.empty((0, 16), device=DEV), none, y=y)[1].shape == (0, 2)
    inv = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device=DEV)
    gone = ue.ue_combine(ctx, torch.empty((0, 16), device=DEV), inv)
    assert not host(gone).any()
    y[0, 3], y[2, 5] = INF, float("nan")
    out = host(ue.ue_combine(ctx, y, inv, torch.full((2, 2), 0.5, device=DEV)))
    assert np.isinf(out[0, 3]) and np.isnan(out[1, 5])
    assert np.isfinite(np.delete(out[0], 3)).all() and np.isfinite(np.delete(out[1], 5)).all()
    x = torch.randn((6, 24), device=DEV).bfloat16()
    perm = torch.randperm(12, device=DEV).int().view(6, 2)
    rows = ue.ue_gather_rows(ctx, x, perm)
    back = ue.ue_combine(ctx, rows, perm)
    assert torch.equal(back, (2 * x.float()).bfloat16())
    ctx.close()


def test_combine_past_4_gib():
    """Rows whose offsets do not fit 32 bits."""
    say("combine past 4 GiB")
    T, k, H = 300, 4, 4096
    ctx = ctx_for(8, k, T)
    rows = 600000                                        # 4.9 GB of bf16
    y = torch.zeros((rows, H), dtype=BF16, device=DEV)
    rng = np.random.default_rng(1)
    inv = np.concatenate([rng.integers(rows - 2000, rows, 600), rng.integers(0, 2000, 600)])
    inv = rng.permutation(np.unique(inv))[:T * k]
    inv = np.resize(inv, T * k).reshape(T, k)
    it = dev(inv.astype(np.int32))
    vals = torch.randn((rows // 150, H), device=DEV).bfloat16()
    y[:2000] = vals[:2000]
    y[rows - 2000:] = vals[2000:4000]
    w = torch.rand((T, k), device=DEV)
    out = ue.ue_combine(ctx, y, it, w)
    want = (y[it.long()].double() * w.double()[..., None]).sum(1)
    size = (y[it.long()].double() * w.double()[..., None]).abs().sum(1)
    assert bool(((out.double() - want).abs() <= 6 * U * size + U16 * want.abs()).all())
    first = torch.tensor(np.unique(inv.reshape(-1), return_index=True)[1], device=DEV)
    keep = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    keep[first] = it.view(-1)[first]                     # every row once
    dout = torch.randn((T, H), device=DEV).bfloat16()
    dy = torch.zeros((rows, H), dtype=BF16, device=DEV)
    dy, dw = ue.ue_combine_backward(ctx, dout, keep.view(T, k), w, y, dy=dy)
    t, j = (keep.view(T, k) >= 0).nonzero(as_tuple=True)
    at = keep.view(T, k)[t, j].long()
    assert torch.equal(dy[at], (dout[t].float() * w[t, j][:, None]).bfloat16())
    want = (dout[t].double() * y[at].double()).sum(1)
    size = (dout[t].double() * y[at].double()).abs().sum(1)
    assert bool(((dw[t, j].double() - want).abs() <= (H / 64 + 20) * U * size).all())
    assert int((dy != 0).any(1).sum()) == at.numel()
    ctx.close()


def test_more_than_one_launch_holds():
    """Tokens and rows past what a launch's threads reach: the parts behind the
    first launch are done too."""
    say("combine in parts")
    T = (1 << 25) + 3
    ctx = ue.Context(2, 1, 0, 1, T, device=DEV)
    inv = torch.arange(T, device=DEV, dtype=torch.int32).flip(0).contiguous().view(T, 1)
    y = (torch.arange(T, device=DEV) % 251).bfloat16().view(T, 1)
    out = ue.ue_combine(ctx, y, inv)
    assert torch.equal(out, y.flip(0))
    w = torch.full((T, 1), 2.0, device=DEV)
    dy, dw = ue.ue_combine_backward(ctx, y, inv, w, y)
    assert torch.equal(dy, 2 * y.flip(0))
    assert torch.equal(dw, y.float() * y.flip(0).float())
    del inv, out, w, dy, dw
    say("pack in parts")
    M = (1 << 29) + 5
    x = torch.zeros((M, 1), dtype=BF16, device=DEV)
    at = torch.tensor([0, 1, (1 << 29) - 1, 1 << 29, M - 1], device=DEV)
    x[at, 0] = torch.tensor([1.0, -3.0, 127.0, 5.0, -0.5], device=DEV).bfloat16()
    q, s = ue.ue_pack_rows(ctx, x)
    assert torch.equal(ue.ue_unpack_rows(ctx, q, s), x)
    assert int((q[:, 0] != 0).sum()) == 5
    ctx.close()


# ---- streams and graphs, and the binding's own checks --------------------------------

def test_other_stream_and_graph():
    """Every operator on a stream of its own, then captured and replayed with
    new inputs between the replays, each replay against the eager result."""
    T, E, k, H, I = 50, 16, 4, 64, 48
    ctx = ctx_for(E, k, T)
    g = torch.Generator(device=DEV).manual_seed(1)
    off = torch.tensor([0, 17, 50], dtype=torch.int32, device=DEV)
    dl = torch.rand(2, generator=g, device=DEV)
    slots = torch.tensor([0, 60, 61, 130, 200], dtype=torch.int32, device=DEV)
    inv = torch.randperm(T * k, generator=g, device=DEV).int().view(T, k)
    perm = torch.empty(T * k, dtype=torch.int32, device=DEV)
    perm[inv.view(-1).long()] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    w = torch.rand((T, k), generator=g, device=DEV)
    mix = torch.randn((H, 2 * I), generator=g, device=DEV).bfloat16()

    def step(x, **kw):
        lg = x[:, :E]
        loss, counts, prob = ue.ue_balance(ctx, lg, ids, off, **kw)
        d = ue.ue_balance_backward(ctx, lg, counts, dl, off, **kw)
        q, s = ue.ue_pack_rows(ctx, x, **kw)
        v = ue.ue_unpack_rows(ctx, q, s, **kw)
        gu = ue.ue_gather_rows(ctx, x, inv, **kw)
        gu = torch.cat([gu, gu], 1)[:, :2 * I].contiguous() if not kw else both(gu, kw["stream"])
        h, gq, gs = ue.ue_gated(ctx, gu, **kw)
        dgu, again = ue.ue_gated_backward(ctx, h, gq, gs, **kw)
        dw = ue.ue_weight_grad(ctx, dgu, q, s, slots, perm, k, **kw)
        out = ue.ue_combine(ctx, again, inv, w, **kw)
        dy, dwt = ue.ue_combine_backward(ctx, out, inv, w, again, **kw)
        return [loss, counts, prob, d, q, s, v, h, dgu, again, dw, out, dy, dwt]

    def both(gu, stream):
        with torch.cuda.stream(stream):
            return torch.cat([gu, gu], 1)[:, :2 * I].contiguous()

    x = torch.randn((T, H), generator=g, device=DEV).bfloat16()
    want = [t.clone() for t in step(x)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(x, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    static = x.clone()
    with torch.cuda.stream(side):
        step(static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        res = step(static)
    for n in range(4):
        say("replay", n)
        new = torch.randn((T, H), generator=g, device=DEV).bfloat16()
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res]
        want = step(new)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    ctx.close()


def test_binding_refusals():
    ctx = ctx_for(8, 2, 16)
    x = torch.randn((4, 8), device=DEV)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    one = torch.ones(1, device=DEV)
    counts = torch.zeros((1, 8), dtype=torch.int32, device=DEV)
    q, s = ue.ue_pack_rows(ctx, x)
    h, gq, gs = ue.ue_gated(ctx, x)
    b = x.bfloat16()
    small = torch.zeros(8, dtype=torch.uint8, device=DEV)
    big = ctx_for(8, 2, 600)                 # so many tokens need a workspace
    many, many_ids = torch.randn((600, 8), device=DEV), ids[:1].repeat(600, 1)
    for err, call in [
            (TypeError, lambda: ue.ue_balance(ctx, x.half(), ids)),
            (ValueError, lambda: ue.ue_balance(ctx, x[:, :7], ids)),
            (ValueError, lambda: ue.ue_balance(ctx, x, ids[:3])),
            (TypeError, lambda: ue.ue_balance(ctx, x, ids.long())),
            (TypeError, lambda: ue.ue_balance(ctx, x, ids, off.long())),
            (ValueError, lambda: ue.ue_balance(ctx, x, ids, [0, 4])),
            (ValueError, lambda: ue.ue_balance(ctx, x, ids, score="tanh")),
            (ValueError, lambda: ue.ue_balance(big, many, many_ids, workspace=small)),
            (ValueError, lambda: ue.ue_balance(ctx, x.cpu(), ids)),
            (ue.UEError, lambda: ue.ue_balance(ctx, torch.randn((17, 8), device=DEV),
                                               torch.zeros((17, 2), dtype=torch.int32, device=DEV))),
            (ValueError, lambda: ue.ue_balance_backward(ctx, x, counts, one, accumulate=True)),
            (ValueError, lambda: ue.ue_balance_backward(ctx, x, counts, torch.ones(2, device=DEV))),
            (ValueError, lambda: ue.ue_balance_backward(ctx, x, counts, one, dlogits=x[:3])),
            (TypeError, lambda: ue.ue_balance_backward(ctx, x, counts, one, dlogits=b)),
            (TypeError, lambda: ue.ue_pack_rows(ctx, x.half())),
            (ValueError, lambda: ue.ue_pack_rows(ctx, x.t())),
            (ValueError, lambda: ue.ue_pack_rows(ctx, x, q=q)),
            (ValueError, lambda: ue.ue_unpack_rows(ctx, q, s[:3])),
            (ValueError, lambda: ue.ue_unpack_rows(ctx, q, None)),
            # packed rows that stop before their block does
            (ValueError, lambda: ue.ue_unpack_rows(ctx, torch.zeros((4, 8), dtype=torch.int8, device=DEV), s)),
            (ValueError, lambda: ue.ue_gated(ctx, x[:, :7])),
            (ValueError, lambda: ue.ue_gated(ctx, x, h=x[:, :3])),
            (ValueError, lambda: ue.ue_gated(ctx, x, q=gq)),
            (ValueError, lambda: ue.ue_gated_backward(ctx, h, q, s)),
            (ValueError, lambda: ue.ue_gated_backward(ctx, h[:3], gq, gs)),
            (TypeError, lambda: ue.ue_weight_grad(ctx, x, b)),
            (TypeError, lambda: ue.ue_weight_grad(ctx, b, x)),
            (ue.UEError, lambda: ue.ue_weight_grad(ctx, b, b[:3])),
            (ValueError, lambda: ue.ue_weight_grad(ctx, b, b, accumulate=True)),
            (ValueError, lambda: ue.ue_weight_grad(ctx, b, b, out=torch.empty((2, 8, 8), device=DEV))),
            (TypeError, lambda: ue.ue_weight_grad(ctx, b, b, out=torch.empty((1, 8, 8), device=DEV).bfloat16())),
            (ValueError, lambda: ue.ue_weight_grad(ctx, b, b, index=off)),
            (ValueError, lambda: ue.ue_combine(ctx, x, ids[:, :1].contiguous().view(-1)[:3])),
            (ValueError, lambda: ue.ue_combine(ctx, x, ids, torch.ones((3, 2), device=DEV))),
            (ValueError, lambda: ue.ue_combine(ctx, x, ids, add=x[:3])),
            (TypeError, lambda: ue.ue_combine(ctx, x, ids, add=b)),
            (ValueError, lambda: ue.ue_combine_backward(ctx, x[:3], ids)),
            (ValueError, lambda: ue.ue_combine_backward(ctx, x, ids, dweights=torch.ones((4, 2), device=DEV))),
            (TypeError, lambda: ue.ue_combine_backward(ctx, x, ids, y=b))]:
        with pytest.raises(err):
            call()
    big.close()
    ctx.close()
