"""One training step of a mixture-of-experts layer on one MI355X, forward and
backward, with the routing rebalanced for exactly these tokens:

  forward   router -> ue_gate -> ue_rebalance; tokens to dispatch order
            (ue_gather_rows), first product of every slot, ue_gated (which keeps
            gate and up in 8 bits), second product, ue_combine back to the tokens
            (onto the residual); ue_balance for the loss that keeps routing even;
            tokens kept in 8 bits (ue_pack_rows)
  backward  ue_combine_backward, the slots' products the other way,
            ue_gated_backward from what was kept, ue_weight_grad per slot,
            ue_grad_reduce of the replicas' gradients into the masters',
            ue_combine for the tokens' gradient, ue_gate_backward and
            ue_balance_backward onto it for the router's

Replicas of hot experts get their weights by ue_weight_sync, from the plan. The
slots' products are the library's matrix products, slot by slot. The script
prints the losses, the balance and the time of a step.

    python examples/moe_train.py [--tokens 4096] [--hidden 2048] [--inter 1024]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_load_ue_amd as ue  # noqa: E402


class Layer:
    """Router and bf16 experts with fp32 gradients; the weights of all physical
    slots lie in one tensor, natives and spares, so that expert e's master is its
    native slot."""

    def __init__(self, E, R, S, k, H, I, max_tokens, device, seed=0,
                 balance=0.01):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.E, self.k, self.H, self.I, self.balance = E, k, H, I, balance
        self.ctx = ctx = ue.Context(E, R, S, k, max_tokens, device=device,
                                    plan_policy=ue.PLAN_BEST_FIT_ASCENDING,
                                    quota_mode=ue.QUOTA_SEARCH)
        self.rule = dict(score="softmax", renorm=True)
        self.router = torch.randn((E, H), generator=g, device=device) * (1.5 / math.sqrt(H))

        def slots(*shape, std):
            return (torch.randn((ctx.P, *shape), generator=g, device=device) * std).bfloat16()
        self.gate_up = slots(2 * I, H, std=1 / math.sqrt(H))
        self.down = slots(H, I, std=1 / math.sqrt(I))
        self.gate_up_grad = torch.zeros(self.gate_up.shape, device=device)
        self.down_grad = torch.zeros(self.down.shape, device=device)
        # expert e is at home in slot r (N + S) + e mod N
        self.native = [e // ctx.N * (ctx.N + S) + e % ctx.N for e in range(E)]
        mats = ((self.gate_up, self.gate_up_grad), (self.down, self.down_grad))
        table = lambda which, at: [[m[which][p].view(-1) for m in mats] for p in at]  # noqa: E731
        every = range(ctx.P)
        ctx.register_experts([2 * I * H, H * I], table(0, self.native), table(1, self.native),
                             table(0, every), table(1, every))

    def forward(self, x, residual, offsets):
        """(out, losses, what the backward pass needs)"""
        ctx, k = self.ctx, self.k
        logits = x.float() @ self.router.t()
        ids, weights = ue.ue_gate(ctx, logits, **self.rule)
        loss, counts, _ = ue.ue_balance(ctx, logits, ids, offsets)
        r = ue.ue_rebalance(ctx, ids)
        plan = ctx.placement_fields(r["placement"])
        replicas = ue.replica_table(ctx, r["placement"])
        ue.ue_weight_sync(ctx, *replicas)
        inv = r["inv_perm"][0].view(-1, k)
        rows = ue.ue_gather_rows(ctx, x, inv)
        bounds = plan["slot_off"][0].tolist()         # (the products' sizes)
        gu = _slot_products(rows, self.gate_up, bounds)
        h, q, scale = ue.ue_gated(ctx, gu)
        y = _slot_products(h, self.down, bounds)
        out = ue.ue_combine(ctx, y, inv, weights, add=residual)
        tokens = ue.ue_pack_rows(ctx, x)
        saved = dict(logits=logits, ids=ids, weights=weights, counts=counts,
                     offsets=offsets, inv=inv, perm=r["perm"][0], plan=plan,
                     bounds=bounds, replicas=replicas, kept=(q, scale), y=y,
                     tokens=tokens)
        return out, loss, saved

    def backward(self, x, saved, dout):
        """Gradients of the tokens (without the residual's own, which is dout)
        and of the router; the experts' go to their gradient buffers."""
        ctx, k, s = self.ctx, self.k, saved
        slots = s["plan"]["slot_off"][0]
        dy, dweights = ue.ue_combine_backward(ctx, dout, s["inv"], s["weights"], y=s["y"])
        dh = _slot_products(dy, self.down.transpose(1, 2), s["bounds"])
        dgu, h = ue.ue_gated_backward(ctx, dh, *s["kept"])
        ue.ue_weight_grad(ctx, dy, h, offsets=slots, out=self.down_grad)
        ue.ue_weight_grad(ctx, dgu, *s["tokens"], offsets=slots, index=s["perm"],
                          index_div=k, out=self.gate_up_grad)
        # masters += replicas, for the experts that the plan gave any
        ue.ue_grad_reduce(ctx, *s["replicas"])
        drows = _slot_products(dgu, self.gate_up.transpose(1, 2), s["bounds"])
        dlogits = ue.ue_gate_backward(ctx, s["logits"], s["ids"], dweights, **self.rule)
        n = s["offsets"].numel() - 1
        dloss = torch.full((n,), self.balance / n, device=x.device)
        ue.ue_balance_backward(ctx, s["logits"], s["counts"], dloss, s["offsets"],
                               dlogits=dlogits, accumulate=True)
        through_router = (dlogits @ self.router).bfloat16()
        dx = ue.ue_combine(ctx, drows, s["inv"], add=through_router)
        return dx, dlogits.t() @ x.float()


def _slot_products(rows, weights, bounds):
    """rows of slot p times weights[p]^T, slot by slot."""
    out = rows.new_empty((rows.shape[0], weights.shape[1]))
    for p in range(weights.shape[0]):
        a, b = bounds[p], bounds[p + 1]
        if a < b:
            torch.matmul(rows[a:b], weights[p].t(), out=out[a:b])
    return out


def run(tokens=4096, hidden=2048, inter=1024, experts=64, ranks=8, spare=2,
        topk=8, sequences=4, device="cuda:0"):
    device = torch.device(device)
    layer = Layer(experts, ranks, spare, topk, hidden, inter, tokens, device)
    g = torch.Generator(device=device)
    g.manual_seed(1)
    x = torch.randn((tokens, hidden), generator=g, device=device).bfloat16()
    target = torch.randn((tokens, hidden), generator=g, device=device)
    cut = torch.rand(sequences - 1, generator=g, device=device).sort().values
    offsets = torch.cat([cut.new_zeros(1), cut, cut.new_ones(1)])
    offsets = (offsets * tokens).round().int()

    def step():
        out, balance, saved = layer.forward(x, x, offsets)
        apart = out.float() - target
        dout = (2 / apart.numel() * apart).bfloat16()
        dx, drouter = layer.backward(x, saved, dout)
        return dict(out=out, error=apart.square().mean(), balance=balance, saved=saved,
                    dout=dout, dx=dx, drouter=drouter)
    return dict(layer=layer, x=x, target=target, offsets=offsets, step=step, **step())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=1024)
    a = ap.parse_args()
    r = run(a.tokens, a.hidden, a.inter)
    plan = r["saved"]["plan"]
    for name in ("load_before", "load_after"):
        load = plan[name][0].float()
        print(f"{name}: max/mean {float(load.max() / load.mean()):.3f}")
    print(f"error {float(r['error']):.4f}, balance loss per sequence "
          f"{[round(v, 4) for v in r['balance'].tolist()]}")
    for _ in range(3):
        r["step"]()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(10):
        r["step"]()
    end.record()
    end.synchronize()
    print(f"a step takes {begin.elapsed_time(end) / 10:.3f} ms")


if __name__ == "__main__":
    main()
