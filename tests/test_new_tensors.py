"""Outputs that the binding makes are torch.empty's wherever a program can tell:
under dispatch and function modes, in deterministic mode (which fills them), and
on the context's device whichever is current."""
import types

import pytest
import torch
from torch.overrides import TorchFunctionMode
from torch.utils._python_dispatch import TorchDispatchMode

import moe_expert_load_ue_amd as ue

CPU = torch.device("cpu")


class Dispatched(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.seen.append(str(func))
        return func(*args, **(kwargs or {}))


class Called(TorchFunctionMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_function__(self, func, types, args=(), kwargs=None):
        self.seen.append(func)
        return func(*args, **(kwargs or {}))


@pytest.fixture
def short(monkeypatch):
    """The binding on a context of device 0, with a short way that notes its
    use."""
    used = []

    def empty(shape, strides, dtype):
        used.append(shape)
        return torch.empty_strided(shape, strides, dtype=dtype)
    monkeypatch.setattr(ue, "_empty", empty)
    monkeypatch.setattr(ue, "_device", lambda: 0)
    return used


def new(index=0):
    return ue._new((3, 5), torch.float32, types.SimpleNamespace(device=CPU, _index=index), None)


def test_dispatch_modes_see_it(short):
    with Dispatched() as mode:
        t = new()
    assert t.shape == (3, 5) and any("aten.empty" in f for f in mode.seen) and not short


def test_function_modes_see_it(short):
    with Called() as mode:
        new()
    assert torch.empty in mode.seen and not short


def test_deterministic_mode_fills_it(short):
    was = torch.are_deterministic_algorithms_enabled(), torch.is_deterministic_algorithms_warn_only_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        t = new()
    finally:
        torch.use_deterministic_algorithms(was[0], warn_only=was[1])
    assert bool(torch.isnan(t).all()) and not short


def test_another_current_device_is_not_used(short):
    assert new(index=1).device == CPU and not short


def test_otherwise_the_short_way(short):
    assert new().shape == (3, 5)
    assert short == [(3, 5)]


@pytest.mark.gpu
def test_on_the_device():
    ctx = ue.Context(8, 1, 0, 2, 16, device="cuda:0")
    x = torch.randn((9, 40), device="cuda:0")
    with Dispatched() as mode:
        q, s = ue.ue_pack_rows(ctx, x)
    assert sum("aten.empty" in f for f in mode.seen) == 2
    assert bool((ue.ue_unpack_rows(ctx, q, s, out_dtype=torch.float32) - x).abs().max() < 0.05)
    torch.use_deterministic_algorithms(True)
    try:
        t = ue._new((1000, 3), torch.bfloat16, ctx, None)
        assert bool(torch.isnan(t).all())
    finally:
        torch.use_deterministic_algorithms(False)
    ctx.close()
