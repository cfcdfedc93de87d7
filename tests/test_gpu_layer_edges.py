"""The expert layer's operators where they once went wrong, and at values and
sizes that tests/test_gpu_layer.py does not reach. u = 2^-24 and u16 = 2^-8 as
there."""
import numpy as np
import pytest
import torch

import moe_expert_load_ue_amd as ue
from gpu_helpers import say
from oracle import layer as L
from tile_rule import compile_rule

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")
U = 2.0 ** -24
U16 = 2.0 ** -8


def ctx_for(E=8, k=2, T=64):
    return ue.Context(E, 1, 0, k, T, device=DEV)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def one_expert(x, gate, up, down):
    """A layer of one expert, hidden 16 and inter 8: x [T, 16]; channel 0 has
    the given gate and up row (over the first entries of x) and every output
    reads it through `down`; the other channels are zero."""
    w13 = torch.zeros((1, 16, 16))
    w13[0, 0, :len(gate)] = torch.tensor(gate)
    w13[0, 8, :len(up)] = torch.tensor(up)
    w2 = torch.zeros((1, 16, 8))
    w2[0, :, 0] = down
    ctx = ctx_for(1, 1, 64)
    router = torch.zeros((1, 16), dtype=torch.bfloat16, device=DEV)
    ue.ue_register_layer(ctx, router, w13.bfloat16().to(DEV), w2.bfloat16().to(DEV))
    xs = torch.zeros((len(x), 16))
    for t, row in enumerate(x):
        xs[t, :len(row)] = torch.tensor(row)
    out, _, _ = ue.ue_moe_tokens(ctx, xs.bfloat16().to(DEV))
    got = host(out)
    ctx.close()
    return got


# ---- silu ---------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 40])
def test_silu_over_the_whole_range(M):
    """Gated products whose gate is exactly v (1 * 1 * v) and whose up is 1.
    Relative error: the exponential and the reciprocal instruction one ulp (2 u)
    each, four roundings: 8 u. Below -88.72 the exponential overflows and the
    result is -0 where the formula has up to 2.6e-37."""
    low = float(np.finfo(np.float32).max)
    v = np.array([INF, low, 3e38, 2.4e38, 2.3e38, 1e38, 1e20, 200.0, 89.0, 88.0,
                  20.0, 3.0, 1.0, 0.5, 1e-3, 1e-30, 0.0, -0.0, -1e-30, -1e-3,
                  -0.5, -1.0, -3.0, -20.0, -80.0, -86.0, -87.0, -87.4, -87.5,
                  -88.0, -88.6, -88.8, -89.0, -104.0, -200.0, -1e20, -1e38,
                  -2.3e38, -2.4e38, -3e38, -low, -INF, np.nan], np.float32)
    v = np.concatenate([v, np.linspace(-88.7, 88.7, 1000).astype(np.float32)])
    n = v.size
    say("silu", M)
    ctx = ctx_for()
    a = torch.ones((M, 16), dtype=torch.int8, device=DEV)[:, :1]
    w = torch.ones((2 * n, 16), dtype=torch.int8, device=DEV)[:, :1]
    sw = dev(np.concatenate([v, np.ones(n, np.float32)]))
    got = host(ue.ue_matmul_i8(ctx, a, torch.ones(M, device=DEV), w, sw, gated=True,
                               out_dtype=torch.float32))
    ctx.close()
    with np.errstate(all="ignore"):
        d = v.astype(np.float64)
        want = np.where(d > 700, d, d / (1 + np.exp(-d)))
    bad = np.isnan(want)
    assert np.isnan(got[:, bad]).all() and not np.isnan(got[:, ~bad]).any()
    assert (got[:, np.isposinf(want)] == INF).all()
    fin = np.isfinite(want)
    assert np.all(np.abs(got[:, fin] - want[fin]) <= 8 * U * np.abs(want[fin]) + 3e-37)


def test_silu_of_large_gates_in_the_layer():
    """A gate of 2.5e38, one that overflows to infinity, and their negatives."""
    got = one_expert([[1, 0], [1, 1], [-1, 0]], [2.5e38, 3e38], [1e-30], 1.0)
    bf = float(torch.tensor(2.5e38).bfloat16()) * float(torch.tensor(1e-30).bfloat16())
    assert np.all(np.abs(got[0] - bf) <= (U16 + 8 * U) * bf)
    assert (got[1] == INF).all()
    assert (got[2] == 0).all()


# ---- registrations and captured graphs ----------------------------------------------------

def test_graph_outlives_further_registrations():
    """A captured layer is replayed after larger and smaller layers were
    registered in the same context and used: each replay, with inputs of its
    own, equal to the eager result of the layer it was captured with."""
    E, k, T = 16, 4, 12
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)

    def layer(H, I):
        r = lambda *s: (torch.randn(s, generator=gen, device=DEV) / s[-1] ** 0.5).bfloat16()  # noqa: E731
        return r(E, H), r(E, 2 * I, H), r(E, H, I)

    ctx, alone = ctx_for(E, k, 64), ctx_for(E, k, 64)
    first, sizes = layer(64, 32), [(4096, 512), (64, 16), (8192, 64), (32, 64)]
    ue.ue_register_layer(ctx, *first)
    ue.ue_register_layer(alone, *first)
    static = torch.zeros((T, 64), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ue.ue_moe_tokens(ctx, static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        res = ue.ue_moe_tokens(ctx, static)
    for n, (H, I) in enumerate(sizes):
        say("registration", n, H, I)
        other = layer(H, I)
        ue.ue_register_layer(ctx, *other)
        y = torch.randn((T, H), generator=gen, device=DEV).bfloat16()
        before = ue.ue_moe_tokens(ctx, y)
        x = torch.randn((T, 64), generator=gen, device=DEV).bfloat16()
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res]
        for a, b in zip(got, ue.ue_moe_tokens(alone, x)):
            assert torch.equal(a, b)
        # and the layer registered last is as it was
        for a, b in zip(ue.ue_moe_tokens(ctx, y), before):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
    ctx.close()
    alone.close()


def test_registration_uses_a_workspace_again():
    """Layers that fit the workspace there is take no more device memory."""
    E, k = 8, 2
    ctx = ctx_for(E, k, 64)
    mk = lambda H, I: [torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
                       for s in ((E, H), (E, 2 * I, H), (E, H, I))]
    big, small = mk(8192, 1024), mk(8192, 64)
    ue.ue_register_layer(ctx, *big)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(40):
        ue.ue_register_layer(ctx, *small)
        ue.ue_register_layer(ctx, *big)
    assert torch.cuda.mem_get_info()[0] == free
    ctx.close()


# ---- the hidden activations' two halves --------------------------------------------

def test_hidden_activation_that_rounds_past_bf16():
    """h = 181/128 2^63 * 181/128 2^64 = 1.9996 2^127 is finite in fp32 and
    rounds to infinity in bf16: its halves have to add up to it all the same."""
    v = 181 / 128
    got = one_expert([[1], [-1]], [v * 2.0 ** 63], [v * 2.0 ** 64], 2.0 ** -100)
    want = v * v * 2.0 ** 27
    assert np.all(np.abs(got[0] - want) <= (U16 + 16 * U) * want)
    # (a negative gate: silu is -0)
    assert (got[1] == 0).all()
    got = one_expert([[1]], [v * 2.0 ** 63], [-v * 2.0 ** 64], 2.0 ** -100)
    assert np.all(np.abs(got[0] + want) <= (U16 + 16 * U) * want)


# ---- launches of 2^32 threads ------------------------------------------------------------

def test_more_rows_than_one_launch_holds():
    """2^26 + 3 rows of one element: more than 2^32 threads at a wave per row."""
    M = (1 << 26) + 3
    say("quantize rows", M)
    x = torch.zeros((M, 1), device=DEV)
    x[-1], x[0], x[1 << 26], x[12345] = 3.0, -2.0, 0.5, INF
    ctx = ctx_for()
    q = torch.full((M, 16), 7, dtype=torch.int8, device=DEV)
    _, s = ue.ue_quantize_rows(ctx, x, q=q[:, :1])
    at = torch.tensor([M - 1, 0, 1 << 26, 12345, 5, (1 << 26) + 1], device=DEV)
    assert q[at, 0].tolist() == [127, -127, 127, 0, 0, 0]
    assert bool((q[:, 1:] == 0).all())
    want = (x[at, 0] / 127).cpu()
    got = s[at].cpu()
    assert torch.equal(got[[0, 1, 2, 4, 5]].sign(), torch.tensor([1.0, 1, 1, 0, 0]))
    assert torch.equal(got[[0, 2]], want[[0, 2]]) and torch.equal(got[1], -want[1])
    assert bool(got[3].isnan())
    assert int((s != 0).sum()) == 4
    ctx.close()


def test_more_channels_than_one_launch_of_the_row_kernel_holds():
    """One row of 16 times 2^27 + 5 channels: 2 GiB, which the limits allow, but
    2^32 threads at 16 channels a workgroup."""
    N = (1 << 27) + 5
    say("one row, channels", N)
    rng = torch.Generator(device=DEV)
    rng.manual_seed(1)
    a = torch.randint(-127, 128, (1, 16), generator=rng, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, 16), generator=rng, device=DEV, dtype=torch.int8)
    sw = torch.ones(N, device=DEV)
    ctx = ctx_for()
    out = ue.ue_matmul_i8(ctx, a, sw[:1], w, sw, out_dtype=torch.float32)
    for lo in range(0, N, 1 << 24):
        part = (w[lo:lo + (1 << 24)].float() * a.float()).sum(1)     # below 2^24: exact
        assert torch.equal(out[0, lo:lo + (1 << 24)], part)
    ctx.close()


# ---- large tiles in every context ---------------------------------------------------------

def test_large_tiles_in_a_second_context():
    """The LDS of the large tiles is granted per context: the first calls of two
    contexts, each with both output types, plain and gated."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(9)
    a = torch.randint(-127, 128, (4096, 256), generator=gen, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (3072, 256), generator=gen, device=DEV, dtype=torch.int8)
    one = torch.full((4096,), 0.01, device=DEV)
    got = []
    for _ in range(2):
        ctx = ctx_for()
        for gated in (False, True):
            for dtype in (torch.float32, torch.bfloat16):
                got.append(ue.ue_matmul_i8(ctx, a, one, w, one[:3072], gated=gated,
                                           out_dtype=dtype))
        torch.cuda.synchronize()
        ctx.close()
    for i in range(4):
        assert torch.equal(got[i], got[i + 4])


# ---- single rows -----------------------------------------------------------------------

def test_a_single_row_of_any_matrix():
    """One row has no next one, so the distance to it is no condition: rows cut
    out of matrices whose own distance would be refused."""
    ctx = ctx_for(8, 2, 16)
    rng = np.random.default_rng(3)
    wide = torch.full((3, 91), 5, dtype=torch.int8, device=DEV)
    a = torch.empty((1, 91), dtype=torch.int8, device=DEV)
    a.copy_(dev(rng.integers(-127, 128, size=(1, 91)).astype(np.int8)))
    wide[:1] = a
    w = dev(rng.integers(-127, 128, size=(5, 96)).astype(np.int8))[:, :80]
    one = torch.ones(5, device=DEV)
    want = (a[:, :80].double() @ w.double().t()).float()
    say("single rows")
    got = ue.ue_matmul_i8(ctx, wide[:1, :80], one[:1], w, one, out_dtype=torch.float32)
    assert torch.equal(got, want)
    # one channel of a matrix likewise
    got = ue.ue_matmul_i8(ctx, w, one, wide[:1, :80], one[:1], out_dtype=torch.float32)
    assert torch.equal(got, want.t())
    # a row of activations into a row of int8
    x = torch.randn((2, 83), device=DEV)
    q = torch.full((2, 91), 9, dtype=torch.int8, device=DEV)
    ue.ue_quantize_rows(ctx, x[:1, :80], q=q[:1, :80])
    assert torch.equal(q[:1, :80], ue.ue_quantize_rows(ctx, x[:1, :80].contiguous())[0])
    assert bool((q[0, 80:] == 9).all()) and bool((q[1] == 9).all())
    # a token
    router = torch.randn((8, 16), device=DEV).bfloat16()
    gu, dn = torch.randn((8, 32, 16), device=DEV).bfloat16(), torch.randn((8, 16, 16), device=DEV).bfloat16()
    ue.ue_register_layer(ctx, router, gu, dn)
    tok = torch.randn((2, 19), device=DEV).bfloat16()
    got = ue.ue_moe_tokens(ctx, tok[:1, :16])
    want = ue.ue_moe_tokens(ctx, tok[:1, :16].contiguous())
    for g, v in zip(got, want):
        assert torch.equal(g, v)
    ctx.close()


# ---- the softmax's gradient far from the top ------------------------------------------

@pytest.mark.parametrize("E", [60, 64, 128, 200, 256])
def test_softmax_gradient_of_unlikely_experts(E):
    """One expert chosen at logit 0, the others 20 to 85 below, in eighths, so
    that differences to the top are exact. Each gradient is -p_e p_0 g: the
    exponential 2 u, the denominator u and its reciprocal or quotient 3 u (the
    other terms are below 256 e^-20), p_0 g with its factor 4 u, the products
    2 u: 12 u, and 16 u here."""
    rng = np.random.default_rng(E)
    T = 70
    x = -rng.integers(160, 680, size=(T, E)) / 8.0
    top = rng.integers(0, E, size=T)
    x[np.arange(T), top] = 0
    dw = (rng.random((T, 1)) + 0.5).astype(np.float32)
    say("unlikely experts", E)
    ctx = ctx_for(E, 1, T)
    got = host(ue.ue_gate_backward(ctx, dev(x, torch.float32), dev(top.astype(np.int32)),
                                   dev(dw), "softmax", False, 1.5))
    ctx.close()
    p = np.exp(x)
    p /= p.sum(1, keepdims=True)
    p0 = p[np.arange(T), top]
    want = -p * (p0 * dw[:, 0] * 1.5)[:, None]
    # (the chosen expert's is p_0 g times the sum of the others: it cancels)
    rest = np.arange(E)[None, :] != top[:, None]
    assert np.all(np.abs(got - want)[rest] <= 16 * U * np.abs(want)[rest])


# ---- every tile of the int8 product ------------------------------------------------------

@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    f = compile_rule(str(tmp_path_factory.mktemp("rule")))
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    return lambda *a: f(*a, num_cu=cus)


def uneven(rng, M, G, low):
    """Offsets of G groups over M rows, one of them empty, none of the others
    below `low`, the last row in none."""
    n = rng.random(G) + 0.3
    n[G // 2] = 0
    rows = np.floor(n / n.sum() * (M - 1 - low * G)).astype(np.int64) + low
    rows[G // 2] = 0
    rows[-1] += M - 1 - rows.sum()
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


# tile wanted, M, channels out (ungated), groups (0: none), the lengths of K
TILED = [("256x256", 4100, 3001, 0, (16, 128, 129, 256, 300, 500, 1000)),
         ("256x256", 6200, 2040, 7, (100, 384, 1990)),
         ("128x256", 6200, 2040, 7, (2048, 2100, 2303)),
         ("128x128", 1500, 2111, 0, (60, 250, 700)),
         ("128x128", 2500, 2100, 9, (333, 2063)),
         ("64x64", 700, 1100, 0, (128, 129, 512, 600, 1030)),
         ("64x64", 1900, 515, 11, (90, 777)),
         ("32x64", 130, 500, 0, (200, 900)),
         ("32x64", 300, 390, 14, (400,))]


@pytest.mark.parametrize("want,M,N,G,Ks", TILED)
@pytest.mark.parametrize("gated", [False, True])
def test_every_tile_by_value(rule, want, M, N, G, Ks, gated):
    """Plain, gated, indexed (an index out of range among them), both output
    types, rows of the output that are and that are not 16-byte aligned, at
    ends of K inside and between stages, against sums in float64 (exact:
    below 2^53). The roundings as in tests/test_gpu_layer.py: 4 u, gated
    1.5e-5 (gates are below 100 here), bf16 u16 more."""
    rng = np.random.default_rng(M + N + G)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(M)

    def i8(*shape):
        return torch.randint(-128, 128, shape, generator=gen, device=DEV, dtype=torch.int8)

    N = N // 2 if gated else N
    mats = max(G, 1)
    ctx = ctx_for()
    for K in Ks:
        assert rule(M, N, K, mats, gated, G > 0).name == want
        ld = (K + 15) // 16 * 16
        ch = 2 * N if gated else N
        k, rows = 3, M // 2
        w = i8(mats, ch, ld)[:, :, :K]
        sw = (torch.rand((mats, ch), generator=gen, device=DEV) + 0.5) / (73 * K ** 0.5)
        off = uneven(rng, M, G, 1) if G else None
        exp = rng.permutation(mats).astype(np.int32)
        if G:
            exp[1] = -1                                     # a slot without expert
        index = rng.integers(0, rows * k, size=M).astype(np.int32)
        index[rng.integers(0, M, size=3)] = [-1, rows * k, 2 ** 31 - 1]
        for indexed, dtype, pad in ((False, torch.float32, 0), (False, torch.bfloat16, 8 - N % 8),
                                    (True, torch.float32, 4 - N % 4), (True, torch.bfloat16, 3)):
            say("tile", want, M, K, N, G, gated, indexed, dtype, pad)
            a = i8(rows if indexed else M, ld)[:, :K]
            sa = (torch.rand(a.shape[0], generator=gen, device=DEV) + 0.5) / 127
            out = torch.full((M, N + pad), -77.0, dtype=dtype, device=DEV)
            ue.ue_matmul_i8(ctx, a, sa, w if G else w[0], sw if G else sw[0],
                            dev(off) if G else None, dev(exp) if G else None,
                            dev(index) if indexed else None, k, gated, out[:, :N])
            r = torch.arange(M, device=DEV)
            if indexed:
                r = torch.div(dev(index).long(), k, rounding_mode="floor")
            ok = (r >= 0) & (r < a.shape[0])
            av = a[r.clamp(0, a.shape[0] - 1)].double() * ok[:, None]
            sv = sa[r.clamp(0, a.shape[0] - 1)].double()
            bounds = off.tolist() if G else [0, M]
            seen = torch.zeros(M, dtype=torch.bool, device=DEV)
            for g in range(len(bounds) - 1):
                e = int(exp[g]) if G else 0
                lo, hi = bounds[g], bounds[g + 1]
                if e < 0 or lo == hi:
                    continue
                seen[lo:hi] = True
                v = av[lo:hi] @ w[e].double().t()
                v = v * sv[lo:hi, None] * sw[e].double()
                if gated:
                    gt = v[:, :N]
                    assert float(gt.abs().max()) < 100
                    v = gt / (1 + torch.exp(-gt)) * v[:, N:]
                tol = (1.5e-5 if gated else 4 * U) * v.abs() + (1e-30 if gated else 0)
                if dtype == torch.bfloat16:
                    tol = tol + U16 * v.abs()
                assert bool(((out[lo:hi, :N].double() - v).abs() <= tol).all()), (K, g)
            assert bool((out[~seen] == -77).all())
            assert bool((out[:, N:] == -77).all())
            assert int(seen.sum()) > M // 2
    ctx.close()


# ---- the gate's approximate ranks, ties and large calls -------------------------------------

def check_choice(x, bias, k, score, renorm, dtype=torch.float32, rank=None):
    """ids, weights and gradient of one call against the oracle."""
    T, E = x.shape
    ctx = ctx_for(E, k, T)
    lg = dev(x, dtype)
    ids, w = ue.ue_gate(ctx, lg, None if bias is None else dev(bias), score, renorm, 2.5)
    want_ids, want_w = L.gate(x, k, score, bias, renorm, 2.5, rank=rank)
    assert np.array_equal(host(ids), want_ids)
    nan = np.isnan(want_w)
    assert np.array_equal(np.isnan(host(w)), nan)
    err = np.abs(host(w) - want_w)[~nan]
    assert np.all(err <= 5e-6 * np.abs(want_w)[~nan] + 1e-30)
    ctx.close()
    return want_ids


@pytest.mark.parametrize("E,k", [(16, 8), (32, 4), (60, 6), (64, 8), (100, 7), (128, 8),
                                 (200, 8), (256, 8), (256, 1), (300, 8)])
def test_gate_logits_apart_in_the_low_bits_only(E, k):
    """fp32 logits that share their upper 24 bits with others of the row, many
    of them equal: the order by all 32 bits, ties to the lowest id."""
    rng = np.random.default_rng(E)
    base = rng.choice(np.array([1.5, 1.4375, -2.0], np.float32), size=(120, E), p=[.5, .3, .2])
    x = (base.view(np.int32) & ~0xFF) + rng.integers(0, 256, size=base.shape).astype(np.int32)
    x[::3] = (base[::3].view(np.int32) & ~0xFF) + rng.integers(0, 3, size=base[::3].shape).astype(np.int32)
    x = x.astype(np.int32).view(np.float32)
    say("low bits", E, k)
    for renorm in (True, False):
        ids = check_choice(x.astype(np.float64), None, k, "softmax", renorm)
    assert (ids >= 0).all()


@pytest.mark.parametrize("E,k", [(16, 8), (32, 4), (60, 6), (64, 8), (128, 8), (200, 8),
                                 (256, 8), (300, 8), (512, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_sigmoid_ties(E, k, dtype):
    """Sigmoid ranks with exact ties: equal logits (with equal biases), and
    logits so large that the fp32 score is 1. Different ranks are at least
    1e-4 apart, so fp32 cannot confuse them; every row is live."""
    rng = np.random.default_rng(E + k)
    levels = np.array([-3.0, -1.25, -0.5, 0.0, 0.75, 1.5, 2.5, 30.0, 40.0, 88.0])
    x = rng.choice(levels, size=(90, E))
    x[0] = 0.75                                     # all equal
    x[1] = rng.choice([20.0, 30.0, 100.0], size=E)  # all saturated
    x[2::5][rng.random(x[2::5].shape) < 0.3] = -INF
    biases = np.array([0.0, 0.3, -0.23, 0.0117], np.float32)
    for bias in (None, rng.choice(biases, size=E)):
        b = np.zeros(E, np.float32) if bias is None else bias
        # the rank as it is defined: in fp32
        p = np.where(x > 17.5, 1.0, L._sigmoid(x)).astype(np.float32)
        rank = (p + b).astype(np.float32)
        u = np.unique(rank)
        near = np.diff(u.astype(np.float64))
        # p rounds within u of its value whoever computes it: ranks of one
        # level and bias are taken as equal, others must be apart
        assert near[near > 1e-6].min() > 1e-4 and (near[near <= 1e-6]).size == 0
        say("sigmoid ties", E, k, dtype, bias is not None)
        for renorm in (True, False):
            ids = check_choice(x, bias, k, "sigmoid", renorm, dtype, rank)
        assert (ids >= 0).mean() > 0.9
        assert ids[0].tolist() == (np.argsort(-b, kind="stable")[:k]).tolist()


@pytest.mark.parametrize("E", [32, 60, 64, 128, 200, 256, 300])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_infinities_and_nan_beside_ordinary_rows(E, score, dtype):
    """Rows with +inf, -inf, NaN, the lowest value, all of one kind, between
    ordinary rows of the same wave, which keep their results."""
    rng = np.random.default_rng(E)
    T, k = 96, 8
    x = np.stack([rng.permutation(np.arange(E)) for _ in range(T)]) * (12.0 / E) - 6
    x = torch.from_numpy(x).to(dtype).double().numpy()
    if score == "sigmoid":
        # apart by more than fp32 scores can confuse, or equal (in bf16)
        p = np.sort(L._sigmoid(x), axis=1)
        gap = np.diff(p, axis=1)
        assert gap[gap > 0].min() > 1e-6
    low = float(torch.finfo(dtype).min)
    x[3, 5] = INF
    x[8, [2, 9, 30]] = INF
    x[13] = -INF
    x[14, :-2] = -INF
    x[21, 7] = np.nan
    x[22] = np.nan
    x[30] = low
    x[31, ::2] = low
    x[40, 1], x[40, 3] = INF, np.nan
    x[51] = INF
    x[52, ::3], x[52, 1::3] = -INF, INF
    say("special rows", E, score, dtype)
    rank = None
    if score == "sigmoid":
        rank = np.where(x > 17.5, 1.0, L._row_scores(x, score))
    for renorm in (True, False):
        check_choice(x, None, k, score, renorm, dtype, rank)


@pytest.mark.parametrize("E,k,dtype", [(256, 8, torch.float32), (256, 8, torch.bfloat16),
                                       (128, 8, torch.float32), (128, 8, torch.bfloat16),
                                       (200, 6, torch.float32), (60, 6, torch.float32),
                                       (32, 8, torch.bfloat16), (256, 16, torch.bfloat16),
                                       (300, 8, torch.float32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_past_one_trip_of_the_grid(E, k, dtype, score):
    """More tokens than the whole grid takes at once (eight workgroups of four
    waves per CU; a token on 8 lanes, on 16, or on a wave), ragged: equal, bit
    for bit, to the same rows in calls that need one trip, and on a sample to
    the oracle."""
    renorm = k % 4 == 0
    lanes = 64 if E > 256 else 16 if E > 128 or k > 8 else 8
    trip = 8 * 4 * torch.cuda.get_device_properties(0).multi_processor_count * (64 // lanes)
    T = 2 * trip + trip // 3 + 5
    gen = torch.Generator(device=DEV)
    gen.manual_seed(E + k)
    x = (torch.randn((T, E), generator=gen, device=DEV) * 2).to(dtype)
    # a third of the rows needs a second look: logits apart in their low bits
    if dtype == torch.float32:
        x[::3] = (1.0 + torch.randint(0, 64, x[::3].shape, generator=gen, device=DEV) * 2.0 ** -23)
    x[5::11].masked_fill_(torch.rand(x[5::11].shape, generator=gen, device=DEV) < 0.3, -INF)
    x[7::97] = -INF
    bias = torch.randn(E, generator=gen, device=DEV) * 0.1 if score == "sigmoid" else None
    dw = torch.randn((T, k), generator=gen, device=DEV)
    say("past one trip", E, k, dtype, score, T)
    ctx = ctx_for(E, k, T)
    ids, w = ue.ue_gate(ctx, x, bias, score, renorm, 2.5)
    d = ue.ue_gate_backward(ctx, x, ids, dw, score, renorm, 2.5)
    n = trip // 2 + 3
    for lo in range(0, T, n):
        s = slice(lo, min(lo + n, T))
        i2, w2 = ue.ue_gate(ctx, x[s], bias, score, renorm, 2.5)
        d2 = ue.ue_gate_backward(ctx, x[s], i2, dw[s], score, renorm, 2.5)
        assert torch.equal(i2, ids[s]) and torch.equal(w2, w[s]) and torch.equal(d2, d[s]), lo
    # every row: distinct ids, best first, nothing better left out
    xd = x.double()
    rank = xd if score == "softmax" else torch.where(
        xd == -INF, xd, torch.sigmoid(xd) + bias.double())
    got = ids >= 0
    mine = torch.where(got, rank.gather(1, ids.clamp_min(0).long()), -INF)
    best = rank.topk(k, dim=1).values
    slack = 0 if score == "softmax" else 1e-6
    assert bool(((best - mine).nan_to_num(0, 0, 0).abs() <= slack).all())
    assert bool((got == (best > -INF)).all())
    spread = torch.where(got, ids.long(), E + torch.arange(k, device=DEV)).sort(1).values
    assert bool((spread[:, 1:] > spread[:, :-1]).all()) or k == 1
    # weights and gradient of rows from every part, at the choice made
    at = torch.cat([torch.arange(0, 40, device=DEV), torch.arange(trip - 20, trip + 20, device=DEV),
                    torch.arange(2 * trip - 5, 2 * trip + 40, device=DEV),
                    torch.arange(T - 40, T, device=DEV)])
    xs, sel = xd[at].cpu().numpy(), ids[at].cpu().numpy()
    order = np.full(xs.shape, -INF)
    for t in range(len(sel)):
        for j, e in enumerate(sel[t]):
            if e >= 0:
                order[t, e] = k - j
    want_ids, want_w = L.gate(xs, k, score, None, renorm, 2.5, rank=order)
    assert np.array_equal(want_ids, sel)
    assert np.all(np.abs(host(w[at]) - want_w) <= 5e-6 * np.abs(want_w) + 1e-30)
    dws = dw[at].cpu().numpy()
    want = L.gate_backward(xs, sel, dws, score, renorm, 2.5)
    tol = 2e-5 * 2.5 * np.abs(dws).max(1, keepdims=True)
    if dtype == torch.bfloat16:
        tol = tol + U16 * np.abs(want)
    assert np.all(np.abs(host(d[at]) - want) <= tol)
    ctx.close()


# ---- many short rows to int8 -------------------------------------------------------------

@pytest.mark.parametrize("K", [1, 8, 17, 1000, 2040, 2048])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_many_short_rows(K, dtype):
    """2,048 rows or more of up to 2,048 elements take a wave each: to the bit
    as the definition (float32 operations), also from unaligned rows."""
    rng = np.random.default_rng(K)
    M = 2051
    v = (rng.normal(size=(M, K)) * np.exp(rng.normal(size=(M, 1)) * 4)).astype(np.float32)
    v[5] = 0
    v[6] = 1e-45
    v[7, K // 2], v[1030, K - 1], v[2050, 0] = INF, np.nan, -INF
    x = dev(v, dtype)
    say("quantize many", K, dtype)
    ctx = ctx_for()
    q, s = ue.ue_quantize_rows(ctx, x)
    f = x.float().cpu().numpy()
    with np.errstate(all="ignore"):
        fine = np.isfinite(f).all(1)
        top = np.abs(f).max(1)
        inv = np.float32(127) / top
        live = fine & (top > 0) & np.isfinite(inv)
        want = np.zeros((M, K), np.int8)
        want[live] = np.rint(f[live] * inv[live, None]).astype(np.int8)
        ws = np.where(live, top / np.float32(127), np.where(fine, 0, np.nan)).astype(np.float32)
    assert live.sum() == M - 5
    assert np.array_equal(host(q), want)
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    pad = torch.as_strided(q, (M, (K + 15) // 16 * 16), (q.stride(0), 1))[:, K:]
    assert bool((pad == 0).all())
    ld = K + 5
    buf = torch.full((M * ld + 1,), 9.0, dtype=dtype, device=DEV)
    u = buf[1:].view(M, ld)[:, :K]
    u.copy_(x)
    q2, s2 = ue.ue_quantize_rows(ctx, u)
    assert torch.equal(q2, q) and np.array_equal(s2.cpu().numpy(), ws, equal_nan=True)
    ctx.close()


# ---- few tokens of a wide layer ----------------------------------------------------------

@pytest.mark.parametrize("T", [1, 3, 4, 5, 8, 9, 20])
@pytest.mark.parametrize("i8", [False, True])
def test_moe_tokens_of_a_wide_layer(T, i8):
    """A hidden size that gives every CU a workgroup of 16 output channels:
    the second product's instances for up to 4 and up to 8 tokens, and the
    next one. Bounds as in tests/test_gpu_layer.py."""
    E, k, I = 6, 3, 48
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    H = 16 * cus + 32                            # (H + 15) / 16 >= cus
    rng = np.random.default_rng(T)
    bf = lambda v: torch.from_numpy(v).bfloat16()  # noqa: E731
    x = bf(rng.normal(size=(T, H)))
    router = bf(rng.normal(size=(E, H)) * 1.5 / np.sqrt(H))
    if i8:
        w13 = torch.from_numpy(rng.integers(-127, 128, size=(E, 2 * I, H)).astype(np.int8))
        w2 = torch.from_numpy(rng.integers(-127, 128, size=(E, H, I)).astype(np.int8))
        s13 = ((rng.random((E, 2 * I)) + 0.5) / (73 * np.sqrt(H))).astype(np.float32)
        s2 = ((rng.random((E, H)) + 0.5) / (73 * np.sqrt(I))).astype(np.float32)
        w13d = w13.double().numpy() * s13.astype(np.float64)[..., None]
        w2d = w2.double().numpy() * s2.astype(np.float64)[..., None]
    else:
        w13 = bf(rng.normal(size=(E, 2 * I, H)) / np.sqrt(H))
        w2 = bf(rng.normal(size=(E, H, I)) / np.sqrt(I))
        s13 = s2 = None
        w13d, w2d = w13.double().numpy(), w2.double().numpy()
    say("wide layer", T, i8, H)
    ctx = ctx_for(E, k, 64)
    ue.ue_register_layer(ctx, router.to(DEV), w13.to(DEV), w2.to(DEV),
                         None if s13 is None else dev(s13), None if s2 is None else dev(s2))
    xs = x.to(DEV)
    out, ids, w = ue.ue_moe_tokens(ctx, xs)
    again, _, _ = ue.ue_moe_tokens(ctx, xs)
    assert torch.equal(out, again)
    out, ids, w = host(out), host(ids), host(w)
    xd = x.double().numpy()
    logits = xd @ router.double().numpy().T
    # the best k of the 64-bit logits, but for what fp32 sums cannot tell apart
    kth = np.sort(logits, 1)[:, -k]
    at = np.arange(T)[:, None]
    assert np.all(logits[at, ids] >= kth[:, None] - 1e-4)
    p = np.exp(logits[at, ids] - logits.max(1, keepdims=True))
    assert np.all(np.abs(w - p / p.sum(1, keepdims=True)) <= 2e-5)
    want, _, _ = L.moe(xd, router.double().numpy(), w13d, w2d, k, choice=(ids, w))
    assert (np.sort(ids, 1)[:, 1:] > np.sort(ids, 1)[:, :-1]).all() and (ids >= 0).all()
    mag = np.zeros(want.shape)
    for t in range(T):
        for j in range(k):
            gu = np.abs(w13d[ids[t, j]]) @ np.abs(xd[t])
            mag[t] += abs(w[t, j]) * (np.abs(w2d[ids[t, j]]) @ (gu[:I] * (gu[I:] + 1)))
    assert np.all(np.abs(out - want) <= U16 * np.abs(want) + 2e-6 * mag)
    ctx.close()
