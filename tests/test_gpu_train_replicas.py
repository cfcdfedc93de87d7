"""The training example's step when experts are replicated: the spare slots take
rows, their gradients reach the masters, and a second step gives the same bits,
the experts' gradients among them."""
import pytest
import torch

from gpu_helpers import say
from test_gpu_train_step import example, reference

pytestmark = pytest.mark.gpu


def test_spare_slots_take_part_and_steps_repeat():
    say("training step, spare slots")
    r = example().run(1500, 64, 32, 16, 4, 2, 2, 2)
    layer = r["layer"]
    # a skewed router, so that the plan has cause to replicate
    layer.router.mul_(2).add_(0.05 * torch.arange(16, device=r["x"].device)[:, None])
    first = r["step"]()
    plan = first["saved"]["plan"]
    assert int(plan["n_rep"][0]) > layer.E
    spare = torch.ones(layer.ctx.P, dtype=torch.bool)
    spare[torch.tensor(layer.native)] = False
    off = plan["slot_off"][0].cpu()
    rows = (off[1:] - off[:-1])[:layer.ctx.P]
    assert int(rows[spare].sum()) > 0 and int(rows.sum()) == 1500 * 2
    native = torch.tensor(layer.native, device=r["x"].device)
    kept = [t[native].clone() for t in (layer.gate_up_grad, layer.down_grad)]
    want = reference({**r, **first})
    # (5% of the 2-norm: rounding to bf16 and to 8 bits, as the step's own test has it)
    for got, exact in zip(kept, (want["gate_up"], want["down"])):
        assert float((got.double() - exact).norm() / exact.norm()) < 0.05
    second = r["step"]()
    for got, grad in zip(kept, (layer.gate_up_grad, layer.down_grad)):
        assert torch.equal(grad[native], got)
    for key in ("out", "balance", "dx", "drouter"):
        assert torch.equal(second[key], first[key]), key
    layer.ctx.close()
