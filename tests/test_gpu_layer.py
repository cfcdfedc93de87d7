"""The expert layer's operators on the GPU against their 64-bit definitions
(oracle/layer.py): the gate and its gradient, 8-bit rows and products, the
whole layer for a few tokens; their refusals; streams and graph replays.

Tolerances, with u = 2^-24 and u16 = 2^-8 (half the spacing above 1
of fp32's 24 and of bf16's 8 significant bits):
- gate weights: an exponential's argument is off by up to |x - top| u (logits
  here differ by less than 30) and its value by 2 u, on both sides of a
  quotient, plus a sum of at most 100 terms in a tree: under 84 u = 5e-6.
- dlogits: sums and products of such scores times g: 2e-5 of the row's largest
  |scale dw| (every factor of g in the formulas is at most 2); bf16 adds u16.
- quantised rows: the stated fp32 operations, so equal to the bit.
- products: three roundings on an exact sum: 4 u; gated, the exponential of
  a gate below 100 adds up to 2 (100 + 4) u: 1.5e-5; bf16 output adds u16.
- layer: out rounds once (u16); before that, sums of K terms carry a few u of
  the sum of their magnitudes (random signs): 2e-6 of the magnitudes' layer.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_ue_amd as ue
from gpu_helpers import say
from oracle import layer as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")
U16 = 2.0 ** -8


def ctx_for(E=8, k=2, T=64):
    return ue.Context(E, 1, 0, k, T, device=DEV)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


# ---- gate -------------------------------------------------------------------

def gate_logits(rng, T, E, k, score, bias, dtype, masked):
    """Logits whose ranks are either equal (to test ties) or apart by more
    than fp32 scores can confuse."""
    x = rng.normal(size=(T, E)) * 2
    if score == "softmax":
        x = np.round(x * 16) / 16            # many exact ties
    x = torch.from_numpy(x).to(dtype).double().numpy()
    if masked:
        x[rng.random((T, E)) < 0.4] = -INF
        x[::7] = -INF                        # rows with nothing left
        x[3::7, : max(E - 1, 1)] = -INF      # rows with at most one left
    if score == "sigmoid":
        for t in range(T):
            p = L._row_scores(x[t], score) + (0 if bias is None else bias)
            r = np.sort(p[np.isfinite(x[t])])
            if r.size > 1 and np.diff(r).min() < 1e-6:
                x[t] = -INF                  # too close to call: masked
    return x


GATE = [(1, 256, 8), (5, 1, 1), (33, 7, 7), (64, 60, 6), (130, 64, 1),
        (257, 65, 3), (90, 128, 8), (70, 250, 8), (61, 300, 5), (19, 512, 16),
        (9, 1000, 8), (6, 1024, 100), (7, 128, 128), (3, 96, 70)]


@pytest.mark.parametrize("T,E,k", GATE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate(T, E, k, score, dtype):
    rng = np.random.default_rng(T * 1000 + E)
    ctx = ctx_for(E, k, T)
    for renorm, masked in ((True, False), (False, True)):
        say("gate", T, E, k, score, dtype, renorm, masked)
        bias = None
        if score == "sigmoid" and renorm:
            bias = rng.normal(size=E).astype(np.float32) * 0.3
        x = gate_logits(rng, T, E, k, score, bias, dtype, masked)
        dw = rng.normal(size=(T, k)).astype(np.float32)
        lg = dev(x, dtype)
        ids, w = ue.ue_gate(ctx, lg, None if bias is None else dev(bias),
                            score, renorm, 2.5)
        want_ids, want_w = L.gate(x, k, score, bias, renorm, 2.5)
        assert np.array_equal(host(ids), want_ids)
        assert np.all(np.abs(host(w) - want_w) <= 5e-6 * np.abs(want_w) + 1e-30)
        d = ue.ue_gate_backward(ctx, lg, ids, dev(dw), score, renorm, 2.5)
        want = L.gate_backward(x, want_ids, dw, score, renorm, 2.5)
        tol = 2e-5 * 2.5 * np.abs(dw).max(1, keepdims=True)
        if dtype == torch.bfloat16:
            tol = tol + U16 * np.abs(want)
        assert d.dtype == dtype
        assert np.all(np.abs(host(d) - want) <= tol)
        # nothing flows into what was masked out
        assert np.all(host(d)[np.isneginf(x)] == 0)
    ctx.close()


def test_gate_special_values():
    """-0 ties with +0, the type's lowest value is a logit, +inf is the
    largest float, NaN poisons its token's weights and no other's."""
    low = float(np.finfo(np.float32).min)
    x = np.array([[-0.0, 0.0, -1, 0.0, -INF, -2], [low] * 6,
                  [low, low, low, -INF, 3.0, low], [1, np.nan, 3, 2, 0, -1],
                  [INF, 5, INF, 0, 0, -INF], [-INF] * 6, [np.nan] * 6,
                  [-INF, -INF, -INF, -INF, -INF, 1e30]], np.float32)
    for renorm in (True, False):
        ctx = ctx_for(6, 3, 8)
        ids, w = ue.ue_gate(ctx, dev(x), renorm=renorm)
        want_ids, want_w = L.gate(x, 3, renorm=renorm)
        assert np.array_equal(host(ids), want_ids)
        assert np.allclose(host(w), want_w, rtol=5e-6, atol=0, equal_nan=True)
        assert host(ids)[0].tolist() == [0, 1, 3]
        assert host(ids)[5].tolist() == [-1, -1, -1]
        d = host(ue.ue_gate_backward(ctx, dev(x[:3]), ids[:3].contiguous(),
                                     torch.ones((3, 3), device=DEV),
                                     renorm=renorm))
        assert np.isfinite(d).all()
        ctx.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_strides_and_offsets(dtype):
    """Rows apart, not 16-byte aligned, outputs given: the same results."""
    rng = np.random.default_rng(2)
    T, E, k = 37, 256, 8
    x = rng.normal(size=(T, E))
    ctx = ctx_for(E, k, 64)
    base = dev(x, dtype)
    ids, w = ue.ue_gate(ctx, base)
    dw = torch.randn((T, k), device=DEV)
    d = ue.ue_gate_backward(ctx, base, ids, dw)
    for ld, off in ((E + 8, 0), (E + 1, 0), (E + 4, 3)):
        say("gate strides", ld, off)
        buf = torch.full((T * ld + off + 8,), float("nan"), dtype=dtype, device=DEV)
        v = buf[off:off + T * ld].view(T, ld)[:, :E]
        v.copy_(base)
        i2, w2 = ue.ue_gate(ctx, v)
        assert torch.equal(i2, ids) and torch.equal(w2, w)
        g = torch.full((T * ld + off,), 7.0, dtype=dtype, device=DEV)
        gv = g[off:off + T * ld].view(T, ld)[:, :E]
        ue.ue_gate_backward(ctx, v, ids, dw, dlogits=gv)
        assert torch.equal(gv, d)
        assert bool((g[off:off + T * ld].view(T, ld)[:, E:] == 7).all())
    e_ids, e_w = ue.ue_gate(ctx, base[:0])
    assert e_ids.shape == (0, k) and e_w.shape == (0, k)
    ctx.close()


def test_gate_gradient_against_differences():
    """The kernel's own weights, differenced: fp32 scores carry about 1e-7,
    a step of 0.02 brings that to 1e-5 and a truncation of h^2/6 = 7e-5."""
    rng = np.random.default_rng(8)
    T, E, k = 4, 20, 4
    x = rng.permuted(np.tile(np.arange(E) * 0.2, (T, 1)), axis=1).astype(np.float32)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    ctx = ctx_for(E, k, T)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, _ = ue.ue_gate(ctx, dev(x), None, score, renorm)
            d = host(ue.ue_gate_backward(ctx, dev(x), ids, dev(dw), score, renorm))
            h = 0.02
            for e in range(E):
                v = []
                for s in (h, -h):
                    y = x.copy()
                    y[:, e] += np.float32(s)
                    i2, w2 = ue.ue_gate(ctx, dev(y), None, score, renorm)
                    assert torch.equal(i2, ids)     # 0.2 apart: no reordering
                    v.append((host(w2) * dw).sum(1))
                step = (x[:, e] + np.float32(h)) - (x[:, e] + np.float32(-h))
                diff = (v[0] - v[1]) / step
                assert np.all(np.abs(diff - d[:, e]) <= 3e-4 * np.abs(dw).max(1))
    ctx.close()


# ---- 8-bit rows ---------------------------------------------------------------

@pytest.mark.parametrize("M,K", [(1, 1), (3, 15), (5, 16), (2, 17), (7, 1000),
                                 (4, 2048), (3, 8192), (2, 8200), (2, 20001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_rows(M, K, dtype):
    rng = np.random.default_rng(K)
    say("quantize", M, K, dtype)
    x = dev(rng.normal(size=(M, K)) * np.exp(rng.normal(size=(M, 1)) * 4), dtype)
    ctx = ctx_for()
    q, s = ue.ue_quantize_rows(ctx, x)
    want_q, want_s = L.quantize(x.float().cpu().numpy())
    assert np.array_equal(host(q), want_q)
    assert np.array_equal(s.cpu().numpy(), want_s)
    pad = torch.as_strided(q, (M, (K + 15) // 16 * 16), (q.stride(0), 1))[:, K:]
    assert bool((pad == 0).all())
    # rows apart and unaligned
    ld = K + 3
    buf = torch.full((M * ld + 1,), 9.0, dtype=dtype, device=DEV)
    v = buf[1:].view(M, ld)[:, :K]
    v.copy_(x)
    q2, s2 = ue.ue_quantize_rows(ctx, v)
    assert torch.equal(q2, q) and torch.equal(s2, s)
    ctx.close()


def test_quantize_special_rows():
    x = np.zeros((7, 40), np.float32)
    x[1, 3] = INF
    x[2, 39] = np.nan
    x[3, 5] = -INF
    x[4] = 1e-45
    x[5] = np.linspace(-1, 1, 40)
    x[6, 0] = np.finfo(np.float32).max
    ctx = ctx_for()
    q, s = ue.ue_quantize_rows(ctx, dev(x))
    want_q, want_s = L.quantize(x)
    assert np.array_equal(host(q), want_q)
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
    w = dev(np.ones((4, 48), np.int8))[:, :40]
    out = host(ue.ue_matmul_i8(ctx, q, s, w, torch.ones(4, device=DEV)))
    # (the largest float itself rounds to infinity in bf16)
    assert np.isnan(out[1:4]).all() and np.isfinite(out[[0, 4, 5]]).all()
    assert ue.ue_quantize_rows(ctx, dev(x)[:0])[0].shape == (0, 40)
    ctx.close()


# ---- products -------------------------------------------------------------------

def i8_case(rng, rows, K, n_mats, channels):
    ld = (K + 15) // 16 * 16
    # garbage, not zeros, between K and the rows' ends
    a = rng.integers(-128, 128, size=(rows, ld)).astype(np.int8)
    w = rng.integers(-128, 128, size=(n_mats, channels, ld)).astype(np.int8)
    sa = (rng.random(rows) + 0.5).astype(np.float32) / 127
    sw = (rng.random((n_mats, channels)) + 0.5).astype(np.float32) / (73 * np.sqrt(K))
    return a, sa, w, sw.astype(np.float32)


def check_product(got, want, gated, dtype):
    tol = (1.5e-5 if gated else 4 * 2.0 ** -24) * np.abs(want)
    if dtype == torch.bfloat16:
        tol = tol + U16 * np.abs(want)
    if gated:
        tol = tol + 1e-30
    assert np.all(np.abs(got - want) <= tol)


SHAPES = [(1, 1, 1), (1, 7168, 64), (1, 100, 130), (2, 33, 5), (9, 129, 70),
          (16, 128, 128), (17, 2049, 129), (31, 64, 300), (33, 255, 1),
          (64, 1024, 64), (65, 300, 257), (130, 200, 200), (256, 384, 256),
          (300, 1900, 514), (515, 127, 40)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("gated", [False, True])
def test_matmul_i8(M, K, N, gated):
    rng = np.random.default_rng(M * 7 + K)
    a, sa, w, sw = i8_case(rng, M, K, 1, 2 * N if gated else N)
    want = L.matmul_i8(a[:, :K], sa, w[0, :, :K], sw, gated=gated)
    ctx = ctx_for()
    for dtype in (torch.float32, torch.bfloat16):
        say("matmul_i8", M, K, N, gated, dtype)
        out = ue.ue_matmul_i8(ctx, dev(a)[:, :K], dev(sa), dev(w[0])[:, :K],
                              dev(sw), gated=gated, out_dtype=dtype)
        assert out.dtype == dtype
        check_product(host(out), want, gated, dtype)
    ctx.close()


GROUPED = [
    # rows of a, K, N, experts, offsets
    (40, 130, 33, 4, [0, 0, 17, 17, 40]),
    (40, 130, 33, 3, [5, 20, 20, 30]),                 # rows outside groups
    (200, 64, 130, 5, [0, 1, 2, 130, 131, 200]),
    (300, 300, 70, 2, [0, 300, 300]),
    (64, 96, 48, 2, [-5, 32, 1000]),                   # clamped
    (600, 260, 100, 6, [0, 3, 260, 260, 300, 599, 600]),
    (1, 512, 64, 1, [0, 1]),
]


@pytest.mark.parametrize("rows,K,N,E,off", GROUPED)
@pytest.mark.parametrize("gated", [False, True])
def test_matmul_i8_groups(rows, K, N, E, off, gated):
    rng = np.random.default_rng(rows + K)
    a, sa, w, sw = i8_case(rng, rows, K, E, 2 * N if gated else N)
    ctx = ctx_for()
    exp = rng.permutation(E).astype(np.int32)
    exp[-1] = -1 if E > 1 else 0                        # a slot without expert
    o = np.array(off, np.int32)
    k = 3
    index = rng.integers(0, rows * k, size=rows).astype(np.int32)
    index[rng.integers(0, rows)] = -1
    index[rng.integers(0, rows)] = rows * k
    for expert_of, idx in ((None, None), (exp, None), (exp, index)):
        say("matmul_i8 groups", rows, K, N, E, gated, idx is not None)
        want = L.matmul_i8(a[:, :K], sa, w[:, :, :K], sw, o, expert_of, idx, k,
                           gated, fill=-77.0)
        out = torch.full((rows, N), -77.0, device=DEV)
        ue.ue_matmul_i8(ctx, dev(a)[:, :K], dev(sa), dev(w)[:, :, :K], dev(sw),
                        dev(o), None if expert_of is None else dev(expert_of),
                        None if idx is None else dev(idx), k, gated, out)
        got = host(out)
        left = want == -77.0
        assert np.array_equal(got[left], want[left])
        check_product(got[~left], want[~left], gated, torch.float32)
    ctx.close()


def test_matmul_i8_strides():
    """Rows and matrices further apart than they are long; outputs apart."""
    rng = np.random.default_rng(4)
    M, K, N, E = 50, 70, 45, 3
    a = rng.integers(-127, 128, size=(M, 112)).astype(np.int8)
    w = rng.integers(-127, 128, size=(E, N + 2, 96)).astype(np.int8)
    sa = rng.random(M).astype(np.float32)
    sw = rng.random((E, N)).astype(np.float32)
    off = np.array([0, 10, 30, 50], np.int32)
    want = L.matmul_i8(a[:, :K], sa, w[:, :N, :K], sw, off)
    out = torch.full((M, N + 5), 3.0, device=DEV)
    ctx = ctx_for()
    ue.ue_matmul_i8(ctx, dev(a)[:, :K], dev(sa), dev(w)[:, :N, :K], dev(sw),
                    dev(off), out=out[:, :N])
    check_product(host(out)[:, :N], want, False, torch.float32)
    assert bool((out[:, N:] == 3).all())
    ctx.close()


def test_matmul_i8_extremes():
    """Sums past 2^24 and the largest of 8 bits: exact before the scales."""
    K = 65536
    a = np.full((3, K), -128, np.int8)
    a[1] = 127
    w = np.full((2, K), -128, np.int8)
    w[1, ::2] = 127
    ctx = ctx_for()
    one = torch.ones(3, device=DEV)
    out = host(ue.ue_matmul_i8(ctx, dev(a), one, dev(w), one[:2],
                               out_dtype=torch.float32))
    want = a.astype(np.int64) @ w.astype(np.int64).T
    assert np.array_equal(out, want.astype(np.float32).astype(np.float64))
    ctx.close()


# ---- the layer for a few tokens ------------------------------------------------

def layer_case(seed, T, E, k, H, I, i8, score):
    """Weights and inputs whose expert ranks are apart by more than fp32 sums
    of the logits can confuse."""
    rng = np.random.default_rng(seed)
    bf = lambda v: torch.from_numpy(v).bfloat16()  # noqa: E731
    x = bf(rng.normal(size=(T, H)))
    router = bf(rng.normal(size=(E, H)) * 1.5 / np.sqrt(H))
    bias = (rng.normal(size=E) * 0.1).astype(np.float32) if score == "sigmoid" else None
    if i8:
        w13 = torch.from_numpy(rng.integers(-127, 128, size=(E, 2 * I, H)).astype(np.int8))
        w2 = torch.from_numpy(rng.integers(-127, 128, size=(E, H, I)).astype(np.int8))
        s13 = ((rng.random((E, 2 * I)) + 0.5) / (73 * np.sqrt(H))).astype(np.float32)
        s2 = ((rng.random((E, H)) + 0.5) / (73 * np.sqrt(I))).astype(np.float32)
    else:
        w13, w2 = bf(rng.normal(size=(E, 2 * I, H)) / np.sqrt(H)), bf(rng.normal(size=(E, H, I)) / np.sqrt(I))
        s13 = s2 = None
    return x, router, bias, w13, w2, s13, s2


def scaled(w, s):
    w = w.double().numpy()
    return w if s is None else w * s.astype(np.float64)[..., None]


def magnitudes(x, w13, w2, ids, w):
    """The layer of the magnitudes, an upper bound of what is summed."""
    out = np.zeros(x.shape)
    I = w2.shape[2]
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            if ids[t, j] >= 0:
                gu = np.abs(w13[ids[t, j]]) @ np.abs(x[t])
                out[t] += abs(w[t, j]) * (np.abs(w2[ids[t, j]]) @ (gu[:I] * (gu[I:] + 1)))
    return out


MOE = [(1, 8, 2, 64, 32), (1, 16, 8, 256, 128), (2, 4, 4, 80, 48),
       (5, 60, 6, 1104, 368), (16, 8, 2, 128, 64), (17, 6, 5, 144, 80),
       (33, 3, 3, 64, 32), (64, 5, 2, 96, 64), (64, 130, 8, 64, 32),
       (7, 1, 1, 48, 16), (3, 300, 9, 64, 32), (9, 70, 65, 32, 16),
       (12, 20, 3, 2048, 512)]


@pytest.mark.parametrize("T,E,k,H,I", MOE)
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_moe_tokens(T, E, k, H, I, i8, score):
    say("moe", T, E, k, H, I, i8, score)
    renorm = T % 2 == 1
    x, router, bias, w13, w2, s13, s2 = layer_case(T * 31 + E, T, E, k, H, I, i8, score)
    ctx = ctx_for(E, k, T)
    ue.ue_register_layer(ctx, router.to(DEV), w13.to(DEV), w2.to(DEV),
                         None if s13 is None else dev(s13),
                         None if s2 is None else dev(s2),
                         None if bias is None else dev(bias), score, renorm, 1.5)
    out, ids, w = ue.ue_moe_tokens(ctx, x.to(DEV))
    out, ids, w = host(out), host(ids), host(w)
    xd, rd = x.double().numpy(), router.double().numpy()
    logits = xd @ rd.T
    want_ids, want_w = L.gate(logits, k, score, bias, renorm, 1.5)
    p = logits if score == "softmax" else L._sigmoid(logits) + (0 if bias is None else bias)
    for t in range(T):
        # where two ranks among the chosen (and the next) are closer than
        # the fp32 logits' error, the order of those two is open
        r = -np.sort(-p[t])[: k + 1]
        if r.size < 2 or -np.diff(r).max() > 1e-5 * max(1, np.abs(logits).max()):
            assert ids[t].tolist() == want_ids[t].tolist(), t
            assert np.all(np.abs(w[t] - want_w[t]) <= 2e-5 * np.abs(want_w[t]))
    w13d, w2d = scaled(w13, s13), scaled(w2, s2)
    want, _, _ = L.moe(xd, rd, w13d, w2d, k, choice=(ids, w))
    tol = U16 * np.abs(want) + 2e-6 * magnitudes(xd, w13d, w2d, ids, w)
    assert np.all(np.abs(out - want) <= tol)
    # the same again: nothing depends on timing
    again, _, _ = ue.ue_moe_tokens(ctx, x.to(DEV))
    assert np.array_equal(host(again), out)
    ctx.close()


def test_moe_rows_do_not_mix():
    """A token's result is the same alone, in a batch, from strided rows, and
    beside a token of NaN or infinities; masked experts are not used; a
    token with no expert left gives zeros."""
    T, E, k, H, I = 6, 12, 3, 128, 64
    x, router, _, w13, w2, _, _ = layer_case(5, T, E, k, H, I, False, "softmax")
    ctx = ctx_for(E, k, 8)
    big = torch.zeros((E, 2 * I * H + 64), dtype=torch.bfloat16, device=DEV)
    apart = big[:, :2 * I * H].view(E, 2 * I, H)
    apart.copy_(w13)
    args = (router.to(DEV), apart, w2.to(DEV))
    ue.ue_register_layer(ctx, *args)
    xd = x.to(DEV)
    out, ids, w = ue.ue_moe_tokens(ctx, xd)
    for t in range(T):
        say("moe row alone", t)
        o1, i1, w1 = ue.ue_moe_tokens(ctx, xd[t:t + 1])
        assert torch.equal(i1[0], ids[t])
        # another split of the sums: fp32 differences, then one rounding
        assert torch.allclose(o1[0].float(), out[t].float(), rtol=2 * U16, atol=1e-3)
    wide = torch.full((T, H + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + H] = xd
    o2 = torch.full((T, H + 3), 5.0, dtype=torch.bfloat16, device=DEV)
    ue.ue_moe_tokens(ctx, wide[:, 8:8 + H], out=o2[:, :H])
    assert torch.equal(o2[:, :H], out) and bool((o2[:, H:] == 5).all())
    bad = xd.clone()
    bad[2, 7] = float("nan")
    bad[4, 0] = float("inf")
    o3, _, w3 = ue.ue_moe_tokens(ctx, bad)
    assert bool(o3[2].isnan().all()) and bool(w3[2].isnan().all())
    for t in (0, 1, 3, 5):
        assert torch.equal(o3[t], out[t])
    # experts masked by their bias
    bias = torch.zeros(E, device=DEV)
    bias[[0, 3, 4]] = -INF
    ue.ue_register_layer(ctx, *args, bias=bias, score="sigmoid")
    _, i4, _ = ue.ue_moe_tokens(ctx, xd)
    assert not bool(torch.isin(i4, torch.tensor([0, 3, 4], device=DEV)).any())
    bias.fill_(-INF)
    o5, i5, w5 = ue.ue_moe_tokens(ctx, xd)
    assert bool((i5 == -1).all()) and bool((w5 == 0).all()) and bool((o5 == 0).all())
    bias.fill_(-INF)
    bias[7] = 0
    o6, i6, _ = ue.ue_moe_tokens(ctx, xd)
    assert host(i6).tolist() == [[7, -1, -1]] * T and bool((o6 != 0).any())
    assert ue.ue_moe_tokens(ctx, xd[:0])[0].shape == (0, H)
    ctx.close()


# ---- refusals, streams, graphs ----------------------------------------------------

def test_refusals_write_nothing():
    ctx = ctx_for(8, 2, 16)
    logits = torch.randn((4, 8), device=DEV)
    ids = torch.full((4, 2), -9, dtype=torch.int32, device=DEV)
    w = torch.full((4, 2), -9.0, device=DEV)
    lib, h = ue.library(), ctx._h
    P = lambda t: ue._ptr(t)  # noqa: E731

    def gate(*, lg=logits, type=ue.F32, ld=8, T=4, score=0, bias=None, i=ids, wt=w):
        return lib.ue_gate(h, P(lg), type, ld, T, score, 1, 1.0, P(bias), P(i), P(wt), None)
    assert gate(T=17) == -2 and gate(T=-1) == -2 and gate(ld=7) == -2
    assert gate(type=2) == -1 and gate(score=5) == -1 and gate(lg=None) == -1
    assert gate(bias=w) == -1 and gate(i=None) == -1 and gate(wt=None) == -1
    assert "sigmoid" in (gate(bias=w) and ue.ue_last_error(ctx))

    def back(*, type=ue.F32, ld=8, T=4, i=ids, dw=w, d=logits, ldo=8):
        return lib.ue_gate_backward(h, P(logits), type, ld, T, 0, 1, 1.0, P(i), P(dw), P(d), ldo, None)
    before = logits.clone()
    assert back(ldo=7) == -2 and back(i=None) == -1 and back(dw=None) == -1
    assert back(T=17) == -2 and back(type=7) == -1 and back(d=None) == -1

    q = torch.full((4, 16), -9, dtype=torch.int8, device=DEV)
    s = torch.full((4,), -9.0, device=DEV)

    def quant(*, x=logits, type=ue.F32, ldx=8, M=4, K=8, qq=q, ldq=16, sc=s):
        return lib.ue_quantize_rows(h, P(x), type, ldx, M, K, P(qq), ldq, P(sc), None)
    assert quant(K=0) == -2 and quant(K=65537) == -2 and quant(M=-1) == -2
    assert quant(ldx=7) == -2 and quant(ldq=8) == -2 and quant(ldq=24) == -2
    assert quant(type=2) == -1 and quant(x=None) == -1 and quant(sc=None) == -1
    assert quant(qq=q.view(-1)[1:]) == -1

    out = torch.full((4, 4), -9.0, device=DEV)
    mat = torch.ones((4, 16), dtype=torch.int8, device=DEV)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)

    def prod(**kw):
        d = dict(a=P(q), a_scale=P(s), w=P(mat), w_scale=P(s), offsets=None,
                 expert_of=None, index=None, out=P(out), lda=16, ldw=16,
                 w_stride=0, ws_stride=0, ldo=4, a_rows=4, n_mats=1, groups=0,
                 index_div=1, M=4, N=4, K=8, gated=0, out_type=ue.F32)
        d.update(kw)
        p = ue.ue_i8_product(**d)
        return lib.ue_matmul_i8(h, ue.ctypes.byref(p), None)
    assert lib.ue_matmul_i8(h, None, None) == -1
    for bad in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=70000), dict(lda=8),
                dict(lda=24), dict(ldw=20), dict(w_stride=4), dict(ldo=3),
                dict(a_rows=3), dict(n_mats=0), dict(expert_of=P(off)),
                dict(offsets=P(off), groups=-1), dict(index=P(off), index_div=0)):
        assert prod(**bad) == -2, bad
    for bad in (dict(a=None), dict(w=None), dict(w_scale=None), dict(out=None),
                dict(a_scale=None), dict(out_type=2), dict(a=q.data_ptr() + 1)):
        assert prod(**bad) == -1, bad

    x = torch.zeros((4, 16), dtype=torch.bfloat16, device=DEV)
    o = torch.full((4, 16), -9.0, dtype=torch.bfloat16, device=DEV)

    def moe(*, xx=x, ldx=16, T=4, oo=o, ldo=16, i=ids, wt=w):
        return lib.ue_moe_tokens(h, P(xx), ldx, T, P(oo), ldo, P(i), P(wt), None)
    assert moe() == -6
    r = torch.zeros((8, 16), dtype=torch.bfloat16, device=DEV)
    g = torch.zeros((8, 32, 16), dtype=torch.bfloat16, device=DEV)
    dn = torch.zeros((8, 16, 16), dtype=torch.bfloat16, device=DEV)

    def reg(**kw):
        d = dict(router=P(r), bias=None, gate_up=P(g), down=P(dn),
                 gate_up_scale=None, down_scale=None, gate_up_stride=512,
                 down_stride=256, hidden=16, inter=16, weight_type=ue.BF16,
                 score=0, renorm=1, scale=1.0)
        d.update(kw)
        return lib.ue_register_layer(h, ue.ctypes.byref(ue.ue_layer(**d)))
    for bad in (dict(hidden=12), dict(inter=4), dict(inter=0), dict(gate_up_stride=511),
                dict(down_stride=255), dict(hidden=24, weight_type=ue.I8)):
        assert reg(**bad) == -2, bad
    for bad in (dict(router=None), dict(weight_type=ue.F32), dict(weight_type=ue.I8),
                dict(score=2), dict(bias=P(s)), dict(down=dn.data_ptr() + 2)):
        assert reg(**bad) == -1, bad
    assert moe() == -6                       # still none registered
    assert reg() == 0
    assert moe(T=17) == -2 and moe(ldx=8) == -2 and moe(ldx=20) == -2
    assert moe(ldo=8) == -2 and moe(xx=None) == -1 and moe(oo=None) == -1
    assert moe(i=None) == -1 and moe(xx=x.view(-1)[1:]) == -1
    torch.cuda.synchronize()
    assert torch.equal(logits, before)
    for t in (ids, w, q, s, out, o):
        assert bool((t == -9).all())

    # the binding's own checks
    with pytest.raises(TypeError):
        ue.ue_gate(ctx, logits.half())
    with pytest.raises(ValueError):
        ue.ue_gate(ctx, logits[:, :7])
    with pytest.raises(ValueError):
        ue.ue_gate(ctx, logits, score="tanh")
    with pytest.raises(ValueError):
        ue.ue_gate(ctx, logits.t().contiguous().t()[:, :8])
    with pytest.raises(ue.UEError):
        ue.ue_gate(ctx, torch.randn((17, 8), device=DEV))
    with pytest.raises(ValueError):
        # the last row's 16-byte piece is not all there
        a = torch.zeros(2 * 16 + 3, dtype=torch.int8, device=DEV)
        ue.ue_matmul_i8(ctx, torch.as_strided(a, (3, 3), (16, 1)), s[:3], mat[:, :3], s)
    with pytest.raises(ValueError):
        ue.ue_matmul_i8(ctx, q, s, mat[:3], s[:3], gated=True)
    ctx.close()


def test_other_stream_and_graph():
    """Every operator on a stream of its own, then captured and replayed with
    new inputs between the replays, each replay against the eager result."""
    T, E, k, H, I = 9, 16, 4, 64, 32
    x, router, _, w13, w2, s13, s2 = layer_case(1, T, E, k, H, I, True, "softmax")
    ctx = ctx_for(E, k, 16)
    w13, w2, s13, s2 = w13.to(DEV), w2.to(DEV), dev(s13), dev(s2)
    ue.ue_register_layer(ctx, router.to(DEV), w13, w2, s13, s2)
    xs = x.to(DEV)
    dw = torch.randn((T, k), device=DEV)
    off = torch.tensor([0, 3, T], dtype=torch.int32, device=DEV)

    def step(v, **kw):
        lg = v[:, :E].float().contiguous()
        ids, w = ue.ue_gate(ctx, lg, **kw)
        d = ue.ue_gate_backward(ctx, lg, ids, dw, **kw)
        q, s = ue.ue_quantize_rows(ctx, v, **kw)
        y = ue.ue_matmul_i8(ctx, q, s, w13, s13, off, gated=True, **kw)
        o, i2, w2_ = ue.ue_moe_tokens(ctx, v, **kw)
        return [ids, w, d, s, y, o, i2, w2_]

    want = [t.clone() for t in step(xs)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(xs, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    static = xs.clone()
    with torch.cuda.stream(side):
        step(static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        res = step(static)
    for n in range(4):
        say("replay", n)
        new = torch.randn((T, H), device=DEV).bfloat16()
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res]
        want = step(new)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    ctx.close()


def test_matmul_i8_rows_past_4_gib():
    """Indexed rows whose offsets do not fit 32 bits."""
    rng = np.random.default_rng(12)
    rows, lda, K, N = 70000, 65536, 70, 33
    a = torch.zeros((rows, lda), dtype=torch.int8, device=DEV)
    pick = np.array([rows - 1, 0, 65535, 65536, 65537, 69998, 12], np.int32)
    vals = rng.integers(-128, 128, size=(pick.size, K)).astype(np.int8)
    a[dev(pick).long(), :K] = dev(vals)
    sa = torch.ones(rows, device=DEV)
    w = rng.integers(-128, 128, size=(N, 80)).astype(np.int8)
    sw = rng.random(N).astype(np.float32)
    ctx = ctx_for()
    for reps in (1, 40):                 # few rows, and enough for tiles
        say("matmul_i8 past 4 GiB", reps)
        idx = np.tile(pick, reps)
        out = ue.ue_matmul_i8(ctx, a[:, :K], sa, dev(w)[:, :K], dev(sw),
                              index=dev(idx), out_dtype=torch.float32)
        want = np.tile((vals.astype(np.int64) @ w[:, :K].astype(np.int64).T) * sw.astype(np.float64), (reps, 1))
        check_product(host(out), want, False, torch.float32)
    ctx.close()


def test_large_tiles_and_even_odd_groups():
    """Sizes that take each of the tiled kernels (256 and 128 rows high, two
    and three stages, K past several stages and ragged), against integer
    products in float64 on the device (exact: sums below 2^53)."""
    rng = torch.Generator(device=DEV)
    rng.manual_seed(5)

    def i8(*shape):
        return torch.randint(-128, 128, shape, generator=rng, device=DEV, dtype=torch.int8)

    ctx = ctx_for()
    for M, K, N, groups in ((3100, 2100, 3001, None), (1500, 700, 2111, None),
                            (5000, 2064, 1100, [0, 700, 700, 1901, 2501, 3900, 4999]),
                            (6000, 272, 1500, [0, 1301, 1302, 3000, 4700, 6000])):
        say("tiles", M, K, N)
        ld = (K + 15) // 16 * 16
        E = len(groups) - 1 if groups else 1
        a, w = i8(M, ld)[:, :K], i8(E, N, ld)[:, :, :K]
        sa, sw = torch.rand(M, device=DEV), torch.rand((E, N), device=DEV)
        off = None if groups is None else torch.tensor(groups, dtype=torch.int32, device=DEV)
        out = torch.full((M, N), -3.0, device=DEV)
        ue.ue_matmul_i8(ctx, a, sa, w, sw, off, out=out)
        g = groups or [0, M]
        for e in range(len(g) - 1):
            s = slice(g[e], g[e + 1])
            want = (a[s].double() @ w[e].double().t()) * (sa[s].double()[:, None] * sw[e].double())
            assert bool(((out[s].double() - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all())
        assert bool((out[g[-1]:] == -3).all())
    ctx.close()


def test_example_layer():
    """The example's layer of many tokens against its layer of few, and
    against the oracle on one token; the router's gradient against the
    oracle's. The many-token form rounds activations twice to 8 bits: steps of
    max/127, about 4/127 of an RMS, so 0.9% and for the heavier-tailed hidden
    rows up to 3%; 5% bounds their sum."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.run(tokens=777, hidden=256, inter=128, experts=32, ranks=4, spare=2,
              topk=4, few=16)
    assert r["same_ids"] == 1.0 and r["apart"] < 0.05
    assert r["after"] <= r["before"]
    lay, s = r["layer"], r["saved"]
    x0 = r["x"][:1].double().cpu().numpy()
    gu = scaled(lay.gate_up.cpu(), lay.gate_up_scale.cpu().numpy())
    dn = scaled(lay.down.cpu(), lay.down_scale.cpu().numpy())
    want, _, _ = L.moe(x0, lay.router.double().cpu().numpy(), gu, dn, 4, "sigmoid",
                       lay.bias.double().cpu().numpy(), True, 2.5)
    got = host(r["out"][:1])
    assert np.linalg.norm(got - want) <= 0.05 * np.linalg.norm(want)
    dout = torch.randn((777, 256), generator=torch.Generator().manual_seed(3)).to(DEV)
    grad = host(lay.router_gradient(r["x"], s, dout))
    dw = (s["rows"].double() * dout.double()[:, None, :]).sum(-1).cpu().numpy()
    dl = L.gate_backward(s["logits"].double().cpu().numpy(), s["ids"].cpu().numpy(),
                         dw, "sigmoid", True, 2.5)
    want = dl.T @ r["x"].double().cpu().numpy()
    # fp32 products over 777 tokens: u sqrt(777) of the magnitudes' product
    mag = np.abs(dl).T @ np.abs(r["x"].double().cpu().numpy())
    assert np.all(np.abs(grad - want) <= 2e-5 * mag + 1e-6)
    lay.ctx.close()
