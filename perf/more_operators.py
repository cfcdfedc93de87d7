"""Measured cases of the expert layer's training step.

Four operators, each as a training step calls it:

balance  the loss that keeps routing even, per packed sequence, with the
         assignments of every expert, and the gradient of the router's logits
gated    silu(gate) * up of the experts' first product, which keeps gate and up
         in 8 bits, and its gradient from what was kept (with silu(gate) * up
         made again for the second product's weight gradient)
wgrad    gradient of the experts' matrices, slot by slot in dispatch order, from
         the gradient of the rows and the tokens: kept in 8 bits ("packed") or
         as they are
combine  weighted sum of the experts' rows back to their tokens, and its
         gradients

What is kept in 8 bits has one power of two per row and 32 columns: the smallest
(from 2^-126) whose 127-fold reaches the block's largest magnitude. Every case
runs in a plain form (elementary torch operations in 32 bits) or, with ``own``
set, through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32             # columns that share a power of two

# Sizes: 256 experts, top-8, hidden 7168, intermediate 2048 and 65536 tokens are
# the DeepSeek-V3-sized configuration of this repository's workloads (dsv3), 64
# experts, 4096 tokens its tiny one. The others are generic, odd ones among them.


def listed():
    return [
        # one short microbatch: launches and latency only
        dict(name="balance_small", op="balance", T=256, E=64, k=8, dtype="bf16",
             score="softmax", seqs=1, masked=0, pad=0),
        # one layer and microbatch of dsv3 size, 16 sequences of different lengths
        dict(name="balance_dsv3", op="balance", T=65536, E=256, k=8, dtype="f32",
             score="sigmoid", seqs=16, masked=0, pad=0),
        # short ragged sequences, padding behind them, experts masked out
        dict(name="balance_odd", op="balance", T=3001, E=60, k=6, dtype="f32",
             score="softmax", seqs=9, masked=20, pad=77),
        # the rows of a few sequences: latency
        dict(name="gated_batch", op="gated", M=64, I=2048, dtype="bf16"),
        # half of a dsv3-sized rank's rows
        dict(name="gated_dsv3", op="gated", M=32768, I=2048, dtype="bf16"),
        # nothing is a multiple of a block or a piece
        dict(name="gated_odd", op="gated", M=1021, I=1002, dtype="f32"),
        # few tokens, no size a multiple of a tile, tokens as they are
        dict(name="wgrad_odd", op="wgrad", T=333, E=5, S=1, k=3, N=366, K=1000,
             packed=False),
        # first matrices of the tiny configuration's experts, the hottest ones
        # split over two slots as after a rebalance
        dict(name="wgrad_tiny", op="wgrad", T=4096, E=64, S=8, k=8, N=2048, K=4096,
             packed=True),
        # first matrices of one dsv3-sized rank: four experts and a replica
        dict(name="wgrad_dsv3", op="wgrad", T=4096, E=4, S=1, k=2, N=4096, K=7168,
             packed=True),
        # one token's experts, with the shared expert's output added
        dict(name="combine_token", op="combine", T=1, k=8, H=7168, dtype="bf16",
             add=True, bwd=False, lost=0),
        # a quarter of a dsv3-sized layer and microbatch, forward and backward
        dict(name="combine_dsv3", op="combine", T=16384, k=8, H=7168, dtype="bf16",
             add=False, bwd=True, lost=0),
        # some assignments without a row, fp32, nothing a multiple of a piece
        dict(name="combine_odd", op="combine", T=1021, k=6, H=1002, dtype="f32",
             add=True, bwd=True, lost=13),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("balance", "gated", "wgrad", "combine"))
    dtype = rng.choice(("f32", "bf16"))
    if op == "balance":
        E = _logint(rng, 8, 512)
        T = min(_logint(rng, 1, 131072), 65536 * 256 // E)
        return dict(op=op, T=T, E=E, k=rng.randint(1, 8), dtype=dtype,
                    score=rng.choice(("softmax", "sigmoid")),
                    seqs=min(T, _logint(rng, 1, 64)), masked=rng.choice((0, 0, 7)),
                    pad=rng.choice((0, 0, T // 9)))
    if op == "gated":
        I = _logint(rng, 30, 4096)
        M = min(_logint(rng, 1, 32768), 32768 * 2048 // I)
        return dict(op=op, M=M if dtype == "bf16" else (M + 1) // 2, I=I, dtype=dtype)
    if op == "wgrad":
        E, k = rng.choice((1, 3, 8, 32, 64)), rng.randint(1, 8)
        N, K = _logint(rng, 64, 4096), _logint(rng, 64, 7168)
        T = min(_logint(rng, 8, 8192), 32768 // k)
        T = max(1, min(T, 8192 * 4096 * 7168 // (k * N * K)))
        E = max(1, min(E, 72 * 2048 * 4096 // (N * K)))
        return dict(op=op, T=T, E=E, S=rng.randint(0, min(8, E)), k=min(k, E), N=N, K=K,
                    packed=rng.random() < 0.6)
    k, H = rng.randint(1, 8), _logint(rng, 60, 7168)
    T = min(_logint(rng, 1, 65536), 16384 * 8 * 7168 // (2 * (k + 1) * H))
    return dict(op=op, T=T, k=k, H=H, dtype=dtype, add=rng.random() < 0.5,
                bwd=rng.random() < 0.6, lost=rng.choice((0, 0, 5)))


def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _ue():
    import moe_expert_load_ue_amd as ue
    return ue


def _dispatch(ids, E, S):
    """Slots of assignments [T, k]: one per expert, and for the S hottest a
    second one that takes the odd tokens'. (offsets, perm)"""
    T, k = ids.shape
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    hot = torch.argsort(counts, descending=True, stable=True)[:S]
    second = torch.full((E,), -1, device=DEV)
    second[hot] = E + torch.arange(hot.numel(), device=DEV)
    odd = (torch.arange(T, device=DEV) % 2 == 1)[:, None]
    slots = torch.where(odd & (second[ids] >= 0), second[ids], ids).reshape(-1)
    n = torch.bincount(slots, minlength=E + hot.numel())
    offsets = torch.cat([n.new_zeros(1), n.cumsum(0)]).int()
    return offsets, torch.argsort(slots, stable=True).int()


def _routing(g, T, E, k):
    """Mildly skewed routing (Zipf 0.5), distinct experts per token."""
    lw = -0.5 * torch.log(1.0 + torch.randperm(E, generator=g, device=DEV))
    keys = lw - torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV)))
    return keys.topk(k, dim=1).indices


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=case, ctx=None)
    op = case["op"]
    if op == "balance":
        T, E, k, n = case["T"], case["E"], case["k"], case["seqs"]
        # per-expert offsets: some experts are hot, as in trained routers
        x = _randn(g, T, E, std=1.5) + _randn(g, 1, E)
        if case["masked"]:
            hide = torch.rand((T, E), generator=g, device=DEV) < 0.3
            hide |= (torch.arange(T, device=DEV) % case["masked"] == 1)[:, None]
            x = x.masked_fill(hide, float("-inf"))
        s["logits"] = x.to(_type(case))
        best, ids = s["logits"].float().topk(k, dim=1)
        s["ids"] = torch.where(best > float("-inf"), ids, -1).int()
        # sequences of different lengths one after another, padding behind them
        cut = torch.rand(n - 1, generator=g, device=DEV).sort().values
        ends = torch.cat([cut, cut.new_ones(1)]) * (T - case["pad"])
        s["offsets"] = torch.cat([ends.new_zeros(1), ends]).round().int()
        # a coefficient of 1e-4 to 1e-2, spread over the sequences
        s["dloss"] = (0.5 + torch.rand(n, generator=g, device=DEV)) * 0.01
        if own:
            s["ctx"] = _ue().Context(E, 1, 0, k, T)
    elif op == "gated":
        M, I = case["M"], case["I"]
        # rows of different sizes, as tokens' activations are
        size = torch.exp(_randn(g, M, 1, std=0.5))
        s["gu"] = (_randn(g, M, 2 * I) * size).to(_type(case))
        s["dh"] = _randn(g, M, I, std=1e-3).to(_type(case))
        if own:
            s["ctx"] = _ue().Context(1, 1, 0, 1, M)
    elif op == "wgrad":
        T, E, k, N, K = (case[n] for n in "TEkNK")
        s["offsets"], s["perm"] = _dispatch(_routing(g, T, E, k), E, case["S"])
        s["rows"] = s["offsets"].tolist()
        s["x"] = (_randn(g, T, K) * torch.exp(_randn(g, T, 1, std=0.5))).bfloat16()
        s["dy"] = _randn(g, T * k, N, std=1e-3).bfloat16()
        if own:
            s["ctx"] = _ue().Context(E, 1, 0, k, T)
    else:
        T, k, H = case["T"], case["k"], case["H"]
        E = 8 * k
        perm = torch.argsort(_routing(g, T, E, k).reshape(-1), stable=True)
        inv = torch.empty_like(perm)
        inv[perm] = torch.arange(T * k, device=DEV)
        if case["lost"]:
            # assignments that found no place have no row; the others close up
            gone = torch.arange(T * k, device=DEV) % case["lost"] == 3
            order = torch.argsort(torch.where(gone, T * k, inv), stable=True)
            inv[order] = torch.arange(T * k, device=DEV)
            inv[gone] = -1
        s["inv"] = inv.view(T, k).int()
        rows = int((inv >= 0).sum())
        s["y"] = _randn(g, rows, H).to(_type(case))
        w = torch.rand((T, k), generator=g, device=DEV) + 0.05
        s["weights"] = 2.5 * w / w.sum(1, keepdim=True)
        s["add"] = _randn(g, T, H).to(_type(case)) if case["add"] else None
        s["dout"] = _randn(g, T, H, std=1e-3).to(_type(case)) if case["bwd"] else None
        if own:
            s["ctx"] = _ue().Context(E, 1, 0, k, T)
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


# ---- through the package --------------------------------------------------

def _run_own(s):
    ue = _ue()
    c, ctx, op = s["case"], s["ctx"], s["case"]["op"]
    if op == "balance":
        loss, counts, prob = ue.ue_balance(ctx, s["logits"], s["ids"], s["offsets"],
                                           score=c["score"])
        d = ue.ue_balance_backward(ctx, s["logits"], counts, s["dloss"], s["offsets"],
                                   score=c["score"])
        return dict(loss=loss, counts=counts, prob=prob, dlogits=d)
    if op == "gated":
        h, q, scale = ue.ue_gated(ctx, s["gu"])
        dgu, again = ue.ue_gated_backward(ctx, s["dh"], q, scale)
        return dict(h=h, dgu=dgu, again=again)
    if op == "wgrad":
        x, scale = ue.ue_pack_rows(ctx, s["x"]) if c["packed"] else (s["x"], None)
        return ue.ue_weight_grad(ctx, s["dy"], x, scale, offsets=s["offsets"],
                                 index=s["perm"], index_div=c["k"])
    out = ue.ue_combine(ctx, s["y"], s["inv"], s["weights"], add=s["add"])
    if not c["bwd"]:
        return out
    dy, dw = ue.ue_combine_backward(ctx, s["dout"], s["inv"], s["weights"], y=s["y"])
    return dict(out=out, dy=dy, dweights=dw)


# ---- plain form ------------------------------------------------------------

def _silu(x):
    return x / (1 + torch.exp(-x))


def _scores(logits, score):
    """(p, what the sigmoid's slope leaves of a gradient)"""
    x = logits.float()
    if score == "softmax":
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
        return e / e.sum(1, keepdim=True).clamp_min(1e-37), 1.0
    p = 1 / (1 + torch.exp(-x))
    return p / (p.sum(1, keepdim=True) + 1e-20), 1 / (1 + torch.exp(x))


def _in_blocks(x):
    """x [M, K] as the values its 8-bit form stands for."""
    M, K = x.shape
    pad = -K % BLOCK
    v = torch.nn.functional.pad(x.float(), (0, pad)).view(M, -1, BLOCK)
    top = v.abs().amax(2, keepdim=True)
    # the exponent of the largest magnitude less six, one more above 127/64 of
    # its power of two
    e = (((top.view(torch.int32) + 0x1FFFF) >> 23) - 6).clamp_min(1)
    step = (e << 23).view(torch.float32)
    inverse = ((254 - e) << 23).view(torch.float32)
    return (torch.round(v * inverse) * step).view(M, -1)[:, :K]


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "balance":
        return _balance_plain(s)
    if op == "gated":
        I, t = c["I"], s["gu"].dtype
        g, u = s["gu"][:, :I].float(), s["gu"][:, I:].float()
        h = (_silu(g) * u).to(t)
        g, u, d = _in_blocks(g), _in_blocks(u), s["dh"].float()
        sig = 1 / (1 + torch.exp(-g))
        dg = d * u * sig * (1 + g * (1 - sig))
        dgu = torch.cat([dg, d * g * sig], 1)
        return dict(h=h, dgu=dgu.to(t), again=(_silu(g) * u).to(t))
    if op == "wgrad":
        x = _in_blocks(s["x"]) if c["packed"] else s["x"].float()
        off = s["rows"]
        out = torch.empty((len(off) - 1, c["N"], c["K"]), device=DEV)
        token = s["perm"].long() // c["k"]
        for g in range(len(off) - 1):
            a, b = off[g], off[g + 1]
            out[g] = torch.matmul(s["dy"][a:b].float().t(), x[token[a:b]])
        return out
    return _combine_plain(s)


def _balance_plain(s):
    c, off = s["case"], s["offsets"].long()
    T, E, k = c["T"], c["E"], c["k"]
    seqs = off.numel() - 1
    p, slope = _scores(s["logits"], c["score"])
    at = torch.arange(T, device=DEV)
    # the sequence of each token; those behind the last one go to a spare row
    seq = torch.searchsorted(off[1:].contiguous(), at, right=True)
    n = (off[1:] - off[:-1]).float()
    ids = s["ids"].long()
    place = torch.where(ids >= 0, seq[:, None] * E + ids, seqs * E)
    counts = torch.bincount(place.reshape(-1), minlength=(seqs + 1) * E)[:seqs * E].view(seqs, E)
    total = torch.zeros((seqs + 1, E), device=DEV).index_add_(0, seq, p)[:seqs]
    factor = torch.where(n > 0, E / (k * n * n), 0.0)
    loss = (counts * total).sum(1) * factor
    prob = total / n.clamp_min(1)[:, None]
    inside = (seq < seqs)[:, None]
    mine = seq.clamp_max(seqs - 1)
    cw = counts.float()[mine]
    d = p * (cw - (p * cw).sum(1, keepdim=True)) * slope
    d = torch.where(inside, d * (s["dloss"] * factor)[mine][:, None], 0.0)
    return dict(loss=loss, counts=counts.int(), prob=prob, dlogits=d.to(s["logits"].dtype))


def _combine_plain(s):
    c, inv, t = s["case"], s["inv"].long(), s["y"].dtype
    has = (inv >= 0)[..., None]
    rows = torch.where(has, s["y"][inv.clamp_min(0)].float(), 0.0)
    out = (rows * s["weights"][..., None]).sum(1)
    if s["add"] is not None:
        out = out + s["add"].float()
    if not c["bwd"]:
        return out.to(t)
    d = s["dout"].float()[:, None, :]
    dw = (rows * d).sum(2)
    dy = torch.zeros_like(s["y"])
    dy[inv[has[..., 0]]] = (d * s["weights"][..., None])[has[..., 0]].to(t)
    return dict(out=out.to(t), dy=dy, dweights=dw)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    b = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op == "balance":
        T, E, k, n = case["T"], case["E"], case["k"], case["seqs"]
        # logits and ids in; gradient, counts and means out
        return dict(bytes=2 * T * E * b + 4 * T * k + n * (8 * E + 12), flops=12 * T * E)
    if op == "gated":
        M, I = case["M"], case["I"]
        # gate, up and dh in; both hidden rows and the gradients out; what is
        # kept for the backward pass is written and read
        return dict(bytes=M * I * (7 * b + 4) + M * I // 8, flops=24 * M * I)
    if op == "wgrad":
        T, k, N, K = case["T"], case["k"], case["N"], case["K"]
        G = case["E"] + min(case["S"], case["E"])
        return dict(bytes=2 * T * K + 2 * T * k * N + 4 * T * k + 4 * G * N * K,
                    flops=2 * T * k * N * K)
    T, k, H = case["T"], case["k"], case["H"]
    n = T * k * (H * b + 8) + T * H * b * (2 if case["add"] else 1)
    if case["bwd"]:
        n += T * k * (H * b + 4) + T * H * b
    return dict(bytes=n, flops=T * k * H * (5 if case["bwd"] else 2))


# ---- the definition, in 64 bits ---------------------------------------------

def _sigma(x):
    return torch.sigmoid(x.double())


def _exact_values(x):
    """What the 8-bit form of x stands for: block by block, the power of two
    from the logarithm of the largest magnitude."""
    x = x.double()
    out = torch.empty_like(x)
    for a in range(0, x.shape[1], BLOCK):
        v = x[:, a:a + BLOCK]
        mantissa, e = torch.frexp(v.abs().amax(1, keepdim=True))
        # top = mantissa 2^e with mantissa in [1/2, 1): 127 2^(e-7) is enough
        # for a mantissa of up to 127/128
        e = torch.where(mantissa > 127 / 128, e - 6, e - 7).clamp_min(-126)
        # (from its bits: a power computed on the device may be off in the last one)
        step = ((e.long() + 1023) << 52).view(torch.float64)
        out[:, a:a + BLOCK] = torch.round(v / step) * step
    return out


def _exact_balance(case, s):
    E, k, off = case["E"], case["k"], s["offsets"].tolist()
    x, ids = s["logits"].double(), s["ids"].long()
    alive = x > float("-inf")
    out = dict(loss=[], counts=[], prob=[])
    d = torch.zeros_like(x)
    for i in range(len(off) - 1):
        r = slice(off[i], off[i + 1])
        n = off[i + 1] - off[i]
        chosen = ids[r].reshape(-1)
        c = torch.bincount(chosen[chosen >= 0], minlength=E)
        out["counts"].append(c.int())
        if n == 0:
            out["loss"].append(x.new_zeros(()))
            out["prob"].append(x.new_zeros(E))
            continue
        # the gradient through autograd
        v = torch.where(alive[r], x[r], -1e300).requires_grad_(True)
        if case["score"] == "softmax":
            p = torch.softmax(v, 1) * alive[r]
        else:
            p = torch.sigmoid(v)
            p = p / (p.sum(1, keepdim=True) + 1e-20)
        mean = p.mean(0)
        loss = E * (c.double() / (k * n) * mean).sum()
        (d[r],) = torch.autograd.grad(s["dloss"][i].double() * loss, v)
        out["loss"].append(loss.detach())
        out["prob"].append(mean.detach())
    out = {name: torch.stack(v) for name, v in out.items()}
    return dict(loss=out["loss"], counts=out["counts"], prob=out["prob"], dlogits=d)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "balance":
        return _exact_balance(case, s)
    if op == "gated":
        I = case["I"]
        g, u = s["gu"][:, :I].double(), s["gu"][:, I:].double()
        h = g * _sigma(g) * u
        g, u = _exact_values(g), _exact_values(u)
        d, sig = s["dh"].double(), _sigma(g)
        dg = d * u * (sig + g * sig * (1 - sig))
        return dict(h=h, dgu=torch.cat([dg, d * g * sig], 1), again=g * sig * u)
    if op == "wgrad":
        x = _exact_values(s["x"]) if case["packed"] else s["x"].double()
        off, perm = s["rows"], s["perm"].tolist()
        out = torch.zeros((len(off) - 1, case["N"], case["K"]), device=DEV, dtype=torch.float64)
        for g in range(len(off) - 1):
            m = torch.arange(off[g], off[g + 1], device=DEV)
            if m.numel():
                rows = torch.tensor([perm[i] // case["k"] for i in range(off[g], off[g + 1])],
                                    device=DEV)
                out[g] = torch.matmul(s["dy"][m].double().t().contiguous(), x[rows])
        return out
    T, k, w = case["T"], case["k"], s["weights"].double()
    out = torch.zeros((T, case["H"]), device=DEV, dtype=torch.float64)
    if s["add"] is not None:
        out += s["add"].double()
    dy = torch.zeros_like(s["y"], dtype=torch.float64) if case["bwd"] else None
    dw = torch.zeros((T, k), device=DEV, dtype=torch.float64)
    for j in range(k):
        t = (s["inv"][:, j] >= 0).nonzero(as_tuple=True)[0]
        at = s["inv"][t, j].long()
        out[t] += w[t, j][:, None] * s["y"][at].double()
        if case["bwd"]:
            d = s["dout"][t].double()
            dy[at] = w[t, j][:, None] * d
            dw[t, j] = (d * s["y"][at].double()).sum(1)
    return dict(out=out, dy=dy, dweights=dw) if case["bwd"] else out
