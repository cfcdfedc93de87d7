"""A call of the expert layer's operators on a context of another device than
the current one is refused: the default stream's handle names no device, so the
kernel would run on the current device with the other one's pointers."""
import types

import pytest

import moe_expert_load_ue_amd as ue


def test_other_device_is_refused(monkeypatch):
    monkeypatch.setattr(ue, "_device", lambda: 0)
    monkeypatch.setattr(ue, "_raw_stream", lambda index: 16 * index)
    ctx = types.SimpleNamespace(_index=1)
    with pytest.raises(ValueError, match="current device is 0, the context's 1"):
        ue._on(ctx, None)
    stream = types.SimpleNamespace(cuda_stream=5)
    with pytest.raises(ValueError, match="set_device"):
        ue._on(ctx, stream)
    ctx._index = 0
    assert ue._on(ctx, None) == 0 and ue._on(ctx, stream) == 5
