"""What the layer's example takes and returns, beyond the types that it is run
with."""
import importlib.util
import os

import pytest
import torch

from gpu_helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_router_gradient_takes_any_output_gradient():
    """Any float type and any strides, as a loss's gradient may come: expanded
    from a sum, a transposed view, halves, doubles."""
    say("router gradient's forms")
    tokens, hidden = 333, 192
    r = example().run(tokens=tokens, hidden=hidden, inter=64, experts=16, ranks=4, spare=1, topk=4, few=8)
    layer, x, saved = r["layer"], r["x"], r["saved"]
    g = torch.Generator(device=DEV).manual_seed(2)
    # halves and bf16 hold these, so every form is the same gradient
    base = torch.randint(-8, 9, (tokens, hidden), generator=g, device=DEV).float() / 8
    want = layer.router_gradient(x, saved, base)
    # dots of 192 terms in another order and a sum over 333 tokens: 2 (192 + 333) u
    # of magnitudes that are at most this many times the result's norm
    tol = 1e-3 * float(want.abs().max())
    for dtype in (torch.float16, torch.bfloat16, torch.float64):
        assert float((layer.router_gradient(x, saved, base.to(dtype)) - want).abs().max()) <= tol
    turned = base.t().contiguous().t()
    assert not turned.is_contiguous()
    for d in (turned, turned.half(), torch.cat([base, base], 1)[:, :hidden]):
        assert float((layer.router_gradient(x, saved, d) - want).abs().max()) <= tol
    one = torch.ones((), device=DEV)
    got = layer.router_gradient(x, saved, one.expand(tokens, hidden))
    want = layer.router_gradient(x, saved, torch.ones((tokens, hidden), device=DEV))
    assert float((got - want).abs().max()) <= 1e-3 * float(want.abs().max())
    layer.ctx.close()


def test_what_is_saved_is_a_plain_dictionary():
    say("what the example saves")
    r = example().run(tokens=64, hidden=64, inter=32, experts=16, ranks=4, spare=1, topk=4, few=8)
    saved = r["saved"]
    assert "rows" in saved and saved.get("rows") is saved["rows"]
    assert dict(saved)["rows"].shape == (64, 4, 64)
    assert {"logits", "ids", "rows", "plan", "counts"} <= set(saved)
    r["layer"].ctx.close()
