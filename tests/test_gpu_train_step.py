"""The training step's operators together, as examples/moe_train.py runs them: a
whole step of the layer, its gradients against autograd in float64 at the same
choice of experts.

The step rounds activations to bf16 between its products (half a step is 2^-8)
and takes the backward pass's tokens, gates and ups from 8 bits: a block's step
is at most its largest magnitude / 63.5, 2.1 standard deviations / 63.5 = 0.033
of 32 normal values on average, which rounds them by 0.033 / sqrt(12) = 0.0095 in
the root mean square. Gradients pass two such roundings (the gate's slope, up,
tokens), each of which the products average over many terms: 5% in the 2-norm
bounds them well, and a term that is missing or wrong shows as tens of percent."""
import importlib.util
import os

import pytest
import torch

import moe_expert_load_ue_amd as ue
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "examples", "moe_train.py")
    spec = importlib.util.spec_from_file_location("moe_train_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(r):
    """Loss and gradients of the step by autograd, in float64."""
    layer, ids, off = r["layer"], r["saved"]["ids"].long(), r["offsets"].tolist()
    native = torch.tensor(layer.native, device=r["x"].device)
    leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
    x, router = leaf(r["x"]), leaf(layer.router)
    gu, dn = leaf(layer.gate_up[native]), leaf(layer.down[native])
    logits = x @ router.t()
    w = torch.softmax(logits.gather(1, ids), 1)
    out = r["x"].double()
    for e in range(layer.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        g, u = (x[t] @ gu[e].t()).chunk(2, 1)
        y = (torch.nn.functional.silu(g) * u) @ dn[e].t()
        out = out.index_add(0, t, y * w[t, j][:, None])
    error = (out - r["target"].double()).square().mean()
    p, losses = torch.softmax(logits, 1), []
    for a, b in zip(off, off[1:]):
        n = max(b - a, 1)
        c = torch.bincount(ids[a:b].reshape(-1), minlength=layer.E).double()
        losses.append(layer.E / (layer.k * n * n) * (c * p[a:b].sum(0)).sum())
    balance = torch.stack(losses)
    (error + layer.balance * balance.mean()).backward()
    return dict(out=out.detach(), error=error.detach(), balance=balance.detach(), dx=x.grad,
                drouter=router.grad, gate_up=gu.grad, down=dn.grad)


@pytest.mark.parametrize("tokens,hidden,inter,experts,ranks,spare,topk,sequences",
                         [(777, 256, 96, 32, 4, 2, 4, 3), (96, 64, 48, 16, 8, 1, 2, 1),
                          (2000, 128, 64, 8, 8, 3, 2, 5)])
def test_example_step(tokens, hidden, inter, experts, ranks, spare, topk, sequences):
    say("training step", tokens, hidden, inter, experts)
    r = example().run(tokens, hidden, inter, experts, ranks, spare, topk, sequences)
    layer = r["layer"]
    want = reference(r)

    def apart(got, exact):
        return float((got.double() - exact).norm() / exact.norm())
    assert apart(r["out"], want["out"]) < 0.02
    assert abs(float(r["error"]) / float(want["error"]) - 1) < 0.01
    assert torch.allclose(r["balance"].double(), want["balance"], rtol=1e-4)
    assert apart(r["dx"], want["dx"]) < 0.05
    assert apart(r["drouter"], want["drouter"]) < 0.05
    native = torch.tensor(layer.native, device=r["x"].device)
    assert apart(layer.gate_up_grad[native], want["gate_up"]) < 0.05
    assert apart(layer.down_grad[native], want["down"]) < 0.05
    # the plan spread the load, so some of these gradients were summed from
    # replicas, and a second step gives the same bits
    assert int((r["saved"]["plan"]["slot_cap"][0] > 0).sum()) > 0
    again = r["step"]()
    for key in ("out", "balance", "dx", "drouter"):
        assert torch.equal(again[key], r[key]), key
    layer.ctx.close()


def test_replicas_take_part():
    """A skewed router makes the plan replicate; masters' gradients are whole all
    the same: dW of expert e is that of all its rows, whichever slot they went to."""
    say("training step with replicas")
    m = example()
    r = m.run(1500, 64, 32, 16, 4, 2, 2, 2)
    layer = r["layer"]
    layer.router.mul_(2).add_(0.05 * torch.arange(16, device=r["x"].device)[:, None])
    again = r["step"]()
    plan = again["saved"]["plan"]
    assert int(plan["n_rep"][0]) > layer.E
    want = reference({**r, **again})
    native = torch.tensor(layer.native, device=r["x"].device)
    for got, exact in ((layer.gate_up_grad[native], want["gate_up"]),
                       (layer.down_grad[native], want["down"]), (again["dx"], want["dx"])):
        assert float((got.double() - exact).norm() / exact.norm()) < 0.05
    layer.ctx.close()


def test_two_graphs_of_a_step_do_not_share_workspaces():
    """Two captured steps of the operators that take a workspace, replayed one
    after the other and at once on two streams, against eager results."""
    say("two graphs")
    dev = torch.device("cuda:0")
    T, E, k, N, K, M = 3000, 64, 4, 96, 160, 20000
    g = torch.Generator(device=dev).manual_seed(2)
    ctx = ue.Context(E, 1, 0, k, T, device=dev)
    cases = []
    for _ in range(2):
        x = torch.randn((T, E), generator=g, device=dev)
        cases.append(dict(x=x, ids=x.topk(k, 1).indices.int(),
                          dy=torch.randn((M, N), generator=g, device=dev).bfloat16(),
                          v=torch.randn((M, K), generator=g, device=dev).bfloat16()))

    def step(c):
        return [*ue.ue_balance(ctx, c["x"], c["ids"]), ue.ue_weight_grad(ctx, c["dy"], c["v"])]
    want = [[t.clone() for t in step(c)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    graphs, results = [], []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            step(c)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            results.append(step(c))
        graphs.append(graph)
    for n in range(4):
        for graph, s in zip(graphs, streams):
            if n % 2:
                with torch.cuda.stream(s):
                    graph.replay()
            else:
                graph.replay()
        torch.cuda.synchronize()
        for got, exact in zip(results, want):
            for a, b in zip(got, exact):
                assert torch.equal(a, b), n
    ctx.close()
