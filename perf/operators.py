"""Measured cases of the expert layer's operators.

Three operators, each as a user's program calls it:

gate     expert choice from router logits: scores, the k best experts of each
         token (ties to the lowest id) with their weights, and the gradient of
         the logits ("bwd": a training step's pass, forward and backward)
i8       products in 8-bit integers: activations quantized row by row, times
         int8 matrices with one scale per channel; either one matrix or one
         matrix per group of rows in dispatch order ("experts": the whole
         gated expert of every group, both products)
moe      a whole mixture-of-experts layer for a few tokens: router, choice of
         experts, gated experts and the weighted sum, from bf16 or int8 weights

Every case runs in a plain form (elementary torch operations in 32 bits) or,
with ``own`` set, through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"

# Sizes: 256 experts, top-8, hidden 7168, intermediate 2048 is the
# DeepSeek-V3-sized configuration of this repository's workloads (dsv3);
# 128 experts and hidden 4096 its pipeline configuration; 4096 tokens over 64
# experts its tiny configuration. The others are generic, odd ones among them.


def listed():
    return [
        # one generated token's expert choice: launch and latency only
        dict(name="gate_token", op="gate", T=1, E=256, k=8, dtype="f32",
             score="sigmoid", renorm=True, bwd=False, masked=0),
        # expert choice of one dsv3-sized layer and microbatch
        dict(name="gate_prefill", op="gate", T=65536, E=256, k=8, dtype="f32",
             score="sigmoid", renorm=True, bwd=False, masked=0),
        # training step over a pipeline microbatch, bf16 logits
        dict(name="gate_train", op="gate", T=131072, E=128, k=8, dtype="bf16",
             score="softmax", renorm=False, bwd=True, masked=0),
        # ragged sizes, experts masked out with -inf, some rows wholly
        dict(name="gate_odd", op="gate", T=1021, E=60, k=6, dtype="f32",
             score="softmax", renorm=True, bwd=True, masked=20),
        # one token through an int8 gate-up matrix of dsv3 size
        dict(name="i8_token", op="i8", M=1, K=7168, N=4096),
        # nothing is a multiple of a tile
        dict(name="i8_odd", op="i8", M=333, K=1900, N=1002),
        # a prefill chunk through the same matrix
        dict(name="i8_prefill", op="i8", M=8192, K=7168, N=4096),
        # prefill of the tiny configuration's tokens through int8 experts,
        # the hottest ones split over two slots as after a rebalance
        dict(name="i8_experts", op="experts", T=4096, E=64, S=8, k=8, H=4096,
             I=1024),
        # one generated token through a small layer: latency counts
        dict(name="moe_token", op="moe", T=1, E=64, k=8, H=2048, I=1024,
             weights="bf16", score="softmax"),
        # one generated token through a dsv3-sized layer with int8 experts
        dict(name="moe_token_dsv3", op="moe", T=1, E=256, k=8, H=7168, I=2048,
             weights="i8", score="sigmoid"),
        # a serving batch through a dsv3-sized layer
        dict(name="moe_batch_dsv3", op="moe", T=32, E=256, k=8, H=7168,
             I=2048, weights="bf16", score="sigmoid"),
        # a few drafted tokens, no size a multiple of a tile
        dict(name="moe_odd", op="moe", T=5, E=60, k=6, H=1104, I=368,
             weights="i8", score="softmax"),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gate", "i8", "experts", "moe", "moe", "gate", "i8"))
    if op == "gate":
        E = _logint(rng, 8, 512)
        T = min(_logint(rng, 1, 131072), 65536 * 256 // E)
        return dict(op=op, T=T, E=E, k=rng.randint(1, 8),
                    dtype=rng.choice(("f32", "bf16")),
                    score=rng.choice(("softmax", "sigmoid")),
                    renorm=rng.random() < 0.5, bwd=rng.random() < 0.6,
                    masked=rng.choice((0, 0, 5)))
    if op == "i8":
        return dict(op=op, M=_logint(rng, 1, 8192), K=_logint(rng, 100, 7168),
                    N=_logint(rng, 64, 4096))
    if op == "experts":
        E = rng.choice((8, 16, 33, 64))
        k = rng.randint(1, 8)
        return dict(op=op, T=min(_logint(rng, 16, 4096), 32768 // k), E=E,
                    S=rng.randint(0, 8), k=k,
                    H=16 * _logint(rng, 32, 256), I=16 * _logint(rng, 8, 64))
    E, k = rng.choice((8, 16, 60, 64, 128, 256)), rng.randint(1, 8)
    T = _logint(rng, 1, 64)
    H, I = 16 * _logint(rng, 32, 448), 16 * _logint(rng, 8, 128)
    T = max(1, min(T, 256 * 2048 * 7168 // (k * H * I)))
    return dict(op=op, T=T, E=E, k=k, H=H, I=I,
                weights=rng.choice(("bf16", "i8")),
                score=rng.choice(("softmax", "sigmoid")))


SCALE = 2.5            # factor on the weights (routed scaling)


def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _i8(g, *shape):
    """int8 matrices [..., N, K] and their channel scales: entries of about
    unit variance over K once scaled."""
    w = torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
    s = (0.5 + torch.rand(shape[:-1], generator=g, device=DEV)) / (73.3 * math.sqrt(shape[-1]))
    return w, s


def _ue():
    import moe_expert_load_ue_amd as ue
    return ue


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=case, ctx=None)
    op = case["op"]
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        # per-expert offsets: some experts are hot, as in trained routers
        x = _randn(g, T, E, std=1.5) + _randn(g, 1, E)
        if case["masked"]:
            hide = torch.rand((T, E), generator=g, device=DEV) < 0.3
            hide |= (torch.arange(T, device=DEV) % case["masked"] == 1)[:, None]
            x = x.masked_fill(hide, float("-inf"))
        s["logits"] = x if case["dtype"] == "f32" else x.bfloat16()
        s["bias"] = _randn(g, E, std=0.1) if case["score"] == "sigmoid" else None
        s["dweights"] = _randn(g, T, k) if case["bwd"] else None
        if own:
            s["ctx"] = _ue().Context(E, 1, 0, k, T)
    elif op == "i8":
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = _randn(g, M, K).bfloat16()
        # rows of a matrix start 16-byte aligned
        w, s["w_scale"] = _i8(g, N, (K + 15) // 16 * 16)
        s["w"] = w[:, :K]
        if own:
            s["ctx"] = _ue().Context(1, 1, 0, 1, M)
    elif op == "experts":
        T, E, S, k, H, I = (case[n] for n in "TESkHI")
        s["x"] = _randn(g, T, H).bfloat16()
        # mildly skewed routing (Zipf 0.5), distinct experts per token
        lw = -0.5 * torch.log(1.0 + torch.randperm(E, generator=g, device=DEV))
        keys = lw - torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV)))
        ids = keys.topk(k, dim=1).indices
        # slots: one per expert; the S hottest experts have a second one that
        # takes every other assignment
        counts = torch.bincount(ids.reshape(-1), minlength=E)
        hot = torch.argsort(counts, descending=True, stable=True)[:S]
        second = torch.full((E,), -1, device=DEV)
        second[hot] = E + torch.arange(hot.numel(), device=DEV)
        odd = (torch.arange(T * k, device=DEV).reshape(T, k) // k) % 2 == 1
        slots = torch.where(odd & (second[ids] >= 0), second[ids], ids).reshape(-1)
        G = E + hot.numel()
        n = torch.bincount(slots, minlength=G)
        s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).int()
        s["slot_expert"] = torch.cat([torch.arange(E, device=DEV), hot]).int()
        s["perm"] = torch.argsort(slots, stable=True).int()
        s["most"] = int(n.max())
        s["w13"], s["s13"] = _i8(g, E, 2 * I, H)
        s["w2"], s["s2"] = _i8(g, E, H, I)
        if own:
            s["ctx"] = _ue().Context(E, 1, 0, k, T)
    else:
        T, E, k, H, I = (case[n] for n in "TEkHI")
        s["x"] = _randn(g, T, H).bfloat16()
        s["router"] = _randn(g, E, H, std=1.5 / math.sqrt(H)).bfloat16()
        s["bias"] = _randn(g, E, std=0.1) if case["score"] == "sigmoid" else None
        if case["weights"] == "i8":
            s["w13"], s["s13"] = _i8(g, E, 2 * I, H)
            s["w2"], s["s2"] = _i8(g, E, H, I)
        else:
            s["w13"] = torch.empty((E, 2 * I, H), device=DEV, dtype=torch.bfloat16).normal_(0, 1 / math.sqrt(H), generator=g)
            s["w2"] = torch.empty((E, H, I), device=DEV, dtype=torch.bfloat16).normal_(0, 1 / math.sqrt(I), generator=g)
            s["s13"] = s["s2"] = None
        if own:
            ue = _ue()
            s["ctx"] = ue.Context(E, 1, 0, k, T)
            ue.ue_register_layer(s["ctx"], s["router"], s["w13"], s["w2"],
                                 s["s13"], s["s2"], bias=s["bias"],
                                 score=case["score"], renorm=True, scale=SCALE)
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


# ---- through the package --------------------------------------------------

def _run_own(s):
    ue = _ue()
    c, ctx, op = s["case"], s["ctx"], s["case"]["op"]
    if op == "gate":
        ids, w = ue.ue_gate(ctx, s["logits"], bias=s["bias"], score=c["score"],
                            renorm=c["renorm"], scale=SCALE)
        if not c["bwd"]:
            return dict(ids=ids, weights=w)
        d = ue.ue_gate_backward(ctx, s["logits"], ids, s["dweights"],
                                score=c["score"], renorm=c["renorm"], scale=SCALE)
        return dict(ids=ids, weights=w, dlogits=d)
    if op == "i8":
        q, qs = ue.ue_quantize_rows(ctx, s["x"])
        return ue.ue_matmul_i8(ctx, q, qs, s["w"], s["w_scale"])
    if op == "experts":
        q, qs = ue.ue_quantize_rows(ctx, s["x"])
        h = ue.ue_matmul_i8(ctx, q, qs, s["w13"], s["s13"], offsets=s["offsets"],
                            expert_of=s["slot_expert"], index=s["perm"],
                            index_div=c["k"], gated=True,
                            out_dtype=torch.float32)
        q, qs = ue.ue_quantize_rows(ctx, h)
        return ue.ue_matmul_i8(ctx, q, qs, s["w2"], s["s2"], offsets=s["offsets"],
                               expert_of=s["slot_expert"])
    out, ids, w = ue.ue_moe_tokens(ctx, s["x"])
    return dict(out=out, ids=ids, weights=w)


# ---- plain form ------------------------------------------------------------

def _silu(x):
    return x / (1 + torch.exp(-x))


def _gate(logits, bias, k, score, renorm):
    """(ids, weights, p): the k best experts, -1 where none is left."""
    x = logits.float()
    if score == "softmax":
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
        p = e / e.sum(1, keepdim=True).clamp_min(1e-37)
        choice = x
    else:
        p = 1 / (1 + torch.exp(-x))
        choice = torch.where(torch.isinf(x) & (x < 0), float("-inf"), p + bias)
    best, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    got = best > float("-inf")
    w = torch.where(got, p.gather(1, ids), 0.0)
    if renorm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return torch.where(got, ids, -1).int(), w * SCALE, p


def _gate_backward(ids, p, dw, score, renorm, dtype):
    got = ids >= 0
    at = ids.clamp_min(0).long()
    gk = torch.where(got, dw * SCALE, 0.0)
    ps = torch.where(got, p.gather(1, at), 0.0)
    if renorm:
        n = ps.sum(1, keepdim=True) + 1e-20
        gk = torch.where(got, (gk - (ps / n * gk).sum(1, keepdim=True)) / n, 0.0)
    dp = torch.zeros_like(p).scatter_add_(1, at, gk)
    if score == "softmax":
        d = p * (dp - (p * dp).sum(1, keepdim=True))
    else:
        d = dp * p * (1 - p)
    return d.to(dtype)


def _quant(x):
    """Rows as whole numbers in -127..127 (held in 32 bits) and their scales."""
    x = x.float()
    top = x.abs().amax(1, keepdim=True)
    q = torch.round(x * torch.where(top > 0, 127 / top, 0.0))
    return q, top / 127


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "gate":
        ids, w, p = _gate(s["logits"], s["bias"], c["k"], c["score"], c["renorm"])
        if not c["bwd"]:
            return dict(ids=ids, weights=w)
        return dict(ids=ids, weights=w,
                    dlogits=_gate_backward(ids, p, s["dweights"], c["score"],
                                           c["renorm"], s["logits"].dtype))
    if op == "i8":
        q, qs = _quant(s["x"])
        return (q @ s["w"].float().t() * qs * s["w_scale"]).bfloat16()
    if op == "experts":
        return _experts_plain(s)
    T, k, H, I = (c[n] for n in "TkHI")
    x = s["x"].float()
    ids, w, _ = _gate(x @ s["router"].float().t(), s["bias"], k, c["score"], True)
    flat = ids.reshape(-1).long()
    w13, w2 = s["w13"][flat].float(), s["w2"][flat].float()
    gu = torch.bmm(w13, x[:, None, :].expand(T, k, H).reshape(T * k, H, 1))[..., 0]
    if s["s13"] is not None:
        gu = gu * s["s13"][flat]
    y = torch.bmm(w2, (_silu(gu[:, :I]) * gu[:, I:])[..., None])[..., 0]
    if s["s2"] is not None:
        y = y * s["s2"][flat]
    out = (y.reshape(T, k, H) * w[..., None]).sum(1)
    return dict(out=out.bfloat16(), ids=ids, weights=w)


def _experts_plain(s):
    """Rows of each slot side by side, padded to the longest slot."""
    c = s["case"]
    k, H, I, most = c["k"], c["H"], c["I"], s["most"]
    off, perm, exp = s["offsets"].long(), s["perm"].long(), s["slot_expert"].long()
    G, M = exp.numel(), perm.numel()
    pos = torch.arange(M, device=off.device)
    slot = torch.searchsorted(off[1:].contiguous(), pos, right=True)
    at = slot * most + pos - off[slot]
    q, qs = _quant(s["x"])
    rows = torch.zeros((G * most, H), device=off.device).index_copy_(0, at, q[perm // k])
    w13 = s["w13"].float().transpose(1, 2).contiguous()[exp]
    gu = torch.bmm(rows.view(G, most, H), w13).view(G * most, 2 * I)[at]
    gu = gu * qs[perm // k] * s["s13"][exp[slot]]
    h, hs = _quant(_silu(gu[:, :I]) * gu[:, I:])
    rows = torch.zeros((G * most, I), device=off.device).index_copy_(0, at, h)
    w2 = s["w2"].float().transpose(1, 2).contiguous()[exp]
    y = torch.bmm(rows.view(G, most, I), w2).view(G * most, H)[at]
    return (y * hs * s["s2"][exp[slot]]).bfloat16()


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    if op == "gate":
        T, E, k, b = case["T"], case["E"], case["k"], 4 if case["dtype"] == "f32" else 2
        # logits in; ids and weights out; backward: dweights in, gradient out
        n = T * E * b + T * k * 8
        if case["bwd"]:
            n += T * k * 4 + T * E * b
        return dict(bytes=n, flops=T * E * (10 if case["bwd"] else 4))
    if op == "i8":
        M, K, N = case["M"], case["K"], case["N"]
        return dict(bytes=2 * M * K + N * K + 4 * N + 2 * M * N, flops=2 * M * N * K)
    T, E, k, H, I = (case[n] for n in "TEkHI")
    # distinct experts met by T tokens of k even choices each
    met = E * (1 - (1 - k / E) ** T)
    if op == "experts":
        return dict(bytes=2 * T * H + met * (3 * I * H + 8 * I + 4 * H) + 4 * T * k + 2 * T * k * H,
                    flops=6 * T * k * I * H)
    size = 2 if case["weights"] == "bf16" else 1
    scales = 0 if size == 2 else 8 * I + 4 * H
    return dict(bytes=4 * T * H + 2 * E * H + met * (size * 3 * I * H + scales) + 8 * T * k,
                flops=6 * T * k * I * H + 2 * T * E * H)


# ---- the definition, in 64 bits ---------------------------------------------

def _sigma(x):
    return torch.sigmoid(x.double())


def _exact_choice(x, bias, k, score, renorm):
    """Expert by expert: k rounds of taking the best that is left."""
    x = x.double()
    alive = x > float("-inf")
    if score == "softmax":
        p = torch.softmax(torch.where(alive, x, -1e300), 1) * alive
        rank = x.clone()
    else:
        p = _sigma(x)
        rank = torch.where(alive, p + bias.double(), float("-inf"))
    picks, parts = [], []
    for _ in range(k):
        best = rank.amax(1, keepdim=True)
        i = (rank == best).int().argmax(1, keepdim=True)
        ok = best > float("-inf")
        picks.append(torch.where(ok, i, -1))
        parts.append(torch.where(ok, p.gather(1, i), 0.0))
        rank.scatter_(1, i, float("-inf"))
    ids, w = torch.cat(picks, 1), torch.cat(parts, 1)
    if renorm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return ids, SCALE * w


def _exact_gradient(x, bias, ids, dw, score, renorm):
    """Through autograd in 64 bits, at the given choice."""
    x = x.double().requires_grad_(True)
    alive = (x > float("-inf")).detach()
    if score == "softmax":
        p = torch.softmax(torch.where(alive, x, -1e300), 1) * alive
    else:
        p = torch.sigmoid(torch.where(alive, x, -1e300))
    w = p.gather(1, ids.clamp_min(0)) * (ids >= 0)
    if renorm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    (SCALE * w * dw.double()).sum().backward()
    return x.grad


def _exact_rows(x):
    x = x.double()
    top = x.abs().amax(1, keepdim=True)
    return torch.round(x * (127 / top)), top / 127


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        ids, w = _exact_choice(s["logits"], s["bias"], case["k"], case["score"], case["renorm"])
        got = dict(ids=None, weights=w)
        if case["bwd"]:
            got["dlogits"] = _exact_gradient(s["logits"], s["bias"], ids, s["dweights"],
                                             case["score"], case["renorm"])
        return got
    if op == "i8":
        q, qs = _exact_rows(s["x"])
        return qs * torch.matmul(q, s["w"].double().t()) * s["w_scale"].double()
    if op == "experts":
        off, I = s["offsets"].tolist(), case["I"]
        q, qs = _exact_rows(s["x"])
        y = torch.empty((s["perm"].numel(), case["H"]), device=DEV, dtype=torch.float64)
        for slot, e in enumerate(s["slot_expert"].tolist()):
            a, b = off[slot], off[slot + 1]
            if a == b:
                continue
            t = torch.div(s["perm"][a:b].long(), case["k"], rounding_mode="floor")
            gu = torch.matmul(q[t], s["w13"][e].double().t()) * qs[t] * s["s13"][e].double()
            h, hs = _exact_rows(gu[:, :I] * _sigma(gu[:, :I]) * gu[:, I:])
            y[a:b] = torch.matmul(h, s["w2"][e].double().t()) * hs * s["s2"][e].double()
        return y
    I = case["I"]
    x = s["x"].double()
    ids, w = _exact_choice(torch.matmul(x, s["router"].double().t()), s["bias"], case["k"],
                           case["score"], True)
    out = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        if e < 0:
            continue
        t, j = (ids == e).nonzero(as_tuple=True)
        w13, w2 = s["w13"][e].double(), s["w2"][e].double()
        if s["s13"] is not None:
            w13, w2 = w13 * s["s13"][e].double()[:, None], w2 * s["s2"][e].double()[:, None]
        gu = torch.matmul(x[t], w13.t())
        h = gu[:, :I] * _sigma(gu[:, :I]) * gu[:, I:]
        out[t] += torch.matmul(h, w2.t()) * w[t, j][:, None]
    return dict(out=out, ids=None, weights=w)
