"""One mixture-of-experts layer with int8 experts, both ways this library
computes it, on one MI355X:

- many tokens (prefill, training): router logits -> ue_gate -> ue_rebalance ->
  ue_quantize_rows -> ue_matmul_i8 over the plan's slots (gated, the tokens
  gathered through the dispatch permutation) -> ue_quantize_rows ->
  ue_matmul_i8 -> weighted sum through the inverse permutation (ue_combine);
  and the router's gradient from the weights' (ue_combine_backward,
  ue_gate_backward); examples/moe_train.py has a whole training step;
- a few tokens (decode): ue_register_layer once, then ue_moe_tokens.

Both use the same weights; the script prints how far the two are apart on the
same tokens (they differ by the 8-bit rounding of the activations, which the
few-token layer does not do), the balance the plan reached, and the times.

    python examples/moe_layer.py [--tokens 4096] [--hidden 2048] [--inter 1024]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_load_ue_amd as ue  # noqa: E402


class Layer:
    """Router and int8 experts of one layer on one device, with E/R experts
    per simulated rank and S spare slots each."""

    def __init__(self, E, R, S, k, H, I, max_tokens, device, seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def i8(*shape):
            w = torch.randint(-127, 128, shape, generator=g, device=device,
                              dtype=torch.int8)
            s = (0.5 + torch.rand(shape[:-1], generator=g, device=device))
            return w, s / (73.3 * math.sqrt(shape[-1]))

        self.k = k
        self.router = (torch.randn((E, H), generator=g, device=device) *
                       (1.5 / math.sqrt(H))).bfloat16()
        # a few popular experts, as a trained router has
        self.bias = 0.1 * torch.randn(E, generator=g, device=device)
        self.gate_up, self.gate_up_scale = i8(E, 2 * I, H)
        self.down, self.down_scale = i8(E, H, I)
        self.rule = dict(score="sigmoid", renorm=True, scale=2.5)
        self.ctx = ue.Context(E, R, S, k, max_tokens, device=device,
                              plan_policy=ue.PLAN_BEST_FIT_ASCENDING,
                              quota_mode=ue.QUOTA_SEARCH)
        ue.ue_register_layer(self.ctx, self.router, self.gate_up, self.down,
                             self.gate_up_scale, self.down_scale,
                             bias=self.bias, **self.rule)

    def many(self, x):
        """(out [T, H], what the passes between need)."""
        ctx, k = self.ctx, self.k
        logits = x.float() @ self.router.float().t()
        ids, weights = ue.ue_gate(ctx, logits, bias=self.bias, **self.rule)
        # the routing is exact, so the plan is made for exactly these tokens
        r = ue.ue_rebalance(ctx, ids)
        plan = ctx.placement_fields(r["placement"])
        slots = dict(offsets=plan["slot_off"][0], expert_of=plan["slot_expert"][0])
        q, qs = ue.ue_quantize_rows(ctx, x)
        h = ue.ue_matmul_i8(ctx, q, qs, self.gate_up, self.gate_up_scale,
                            index=r["perm"][0], index_div=k, gated=True,
                            out_dtype=torch.float32, **slots)
        q, qs = ue.ue_quantize_rows(ctx, h)
        y = ue.ue_matmul_i8(ctx, q, qs, self.down, self.down_scale, **slots)
        inv = r["inv_perm"][0].view(-1, k)
        out = ue.ue_combine(ctx, y, inv, weights)
        return out, dict(logits=logits, ids=ids, weights=weights, y=y, inv=inv,
                         rows=y[inv.long()], plan=plan, counts=r["counts"])

    def router_gradient(self, x, saved, dout):
        """Gradient of the router's matrix from that of the output (the part
        that flows through the routing weights). dout: of any float type and
        strides."""
        y = saved["y"]
        if dout.dtype != y.dtype:
            y, dout = y.float(), dout.float()
        _, dw = ue.ue_combine_backward(self.ctx, dout.contiguous(), saved["inv"],
                                       saved["weights"], y=y, with_dy=False)
        dlogits = ue.ue_gate_backward(self.ctx, saved["logits"], saved["ids"], dw,
                                      **self.rule)
        return dlogits.t() @ x.float()

    def few(self, x):
        return ue.ue_moe_tokens(self.ctx, x)


def timed(f, n=20):
    for _ in range(3):
        f()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(n):
        f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / n * 1e3


def run(tokens=4096, hidden=2048, inter=1024, experts=64, ranks=8, spare=2,
        topk=8, few=16, device="cuda:0"):
    device = torch.device(device)
    layer = Layer(experts, ranks, spare, topk, hidden, inter, tokens, device)
    g = torch.Generator(device=device)
    g.manual_seed(1)
    x = torch.randn((tokens, hidden), generator=g, device=device).bfloat16()
    out, saved = layer.many(x)
    dout = torch.randn((tokens, hidden), generator=g, device=device).bfloat16()
    grad = layer.router_gradient(x, saved, dout)
    few_out, few_ids, _ = layer.few(x[:few])
    torch.cuda.synchronize(device)
    load = saved["plan"]["load_after"][0].float()
    native = saved["plan"]["load_before"][0].float()
    a, b = out[:few].float(), few_out.float()
    return dict(layer=layer, x=x, out=out, grad=grad, saved=saved,
                same_ids=float((few_ids == saved["ids"][:few]).float().mean()),
                apart=float((a - b).norm() / b.norm()),
                before=float(native.max() / native.mean()),
                after=float(load.max() / load.mean()))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=1024)
    a = ap.parse_args()
    r = run(a.tokens, a.hidden, a.inter)
    layer, x = r["layer"], r["x"]
    print(f"same experts chosen: {100 * r['same_ids']:.2f}%; outputs apart by "
          f"{r['apart']:.4f} (2-norm); router gradient norm "
          f"{float(r['grad'].norm()):.3f}")
    print(f"max/mean rank load {r['before']:.3f} -> {r['after']:.3f}")
    print(f"{a.tokens} tokens: {timed(lambda: layer.many(x)):.1f} us a pass")
    for n in (1, 8, 64):
        print(f"{n} tokens: {timed(lambda: layer.few(x[:n])):.1f} us a pass")


if __name__ == "__main__":
    main()
