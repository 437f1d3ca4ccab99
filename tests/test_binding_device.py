"""Calls on tensors of a device that is not the current one (CPU only): every call of the layer's forward and of a
training step makes the tensors' device current while libmoe launches, and leaves the caller's current afterwards."""

from types import SimpleNamespace

import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B

T, H, E, K, I, I_S = 6, 16, 4, 2, 8, 24


class FakeTensor:
    """Shape, type and device of a tensor, and no memory."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, SimpleNamespace(type="cuda", index=1)

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)


class FakeLib:
    """Notes the device that is current when a call is made."""

    def __init__(self, state):
        self.state, self.calls = state, []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 64
            self.calls.append((name, self.state.current))
            return 0
        return call


@pytest.fixture()
def lib(monkeypatch):
    state = SimpleNamespace(current=0)
    fake = FakeLib(state)

    class Guard:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, state.current = state.current, self.index

        def __exit__(self, *exc):
            state.current = self.before

    monkeypatch.setattr(B, "load", lambda path=None: fake)
    monkeypatch.setattr(B, "_ptr", lambda t, *a, **k: 0)
    monkeypatch.setattr(B, "_stream", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    fake.real_current = state
    return fake


def fill(monkeypatch, cls, *args):
    """Buffers of a layer without their memory."""
    with monkeypatch.context() as m:
        for name in ("empty", "zeros"):
            m.setattr(torch, name, lambda shape, dtype=None, device=None: FakeTensor(*shape, dtype=dtype))
        return cls(*args, torch.bfloat16, SimpleNamespace(type="cuda", index=1))


@pytest.mark.parametrize("gated", [False, True])
def test_layer_calls_launch_on_the_tensors_device(lib, monkeypatch, gated):
    x, wr, dy = FakeTensor(T, H), FakeTensor(H, E), FakeTensor(T, H, dtype=torch.float32)
    W1, W2 = FakeTensor(E, H, 2 * I), FakeTensor(E, I, H)
    shared = (FakeTensor(H, 2 * I_S), FakeTensor(I_S, H), FakeTensor(H) if gated else None)
    bufs = fill(monkeypatch, B.MoELayerBuffers, T, H, E, K, I, I_S)
    train = fill(monkeypatch, B.MoETrainBuffers, T, H, E, K, I, I_S, gated, False)
    B.moe_layer_train_forward(x, wr, None, W1, W2, K, shared, bufs, train)
    B.moe_layer_backward(dy, x, wr, W1, W2, shared, bufs, train, max_norm=1.0)
    names = [n for n, _ in lib.calls]
    assert names == ["moe_route", "moe_build_scatter", "moe_grouped_swiglu_fc1_save", "moe_grouped_fc2",
                     "moe_gather_combine", "moe_shared_fc1_save", "moe_shared_fc2_save", "moe_scatter_grad",
                     "moe_grouped_fc2_backward", "moe_grouped_fc1_backward", "moe_route_backward",
                     "moe_shared_fc2_backward", "moe_shared_fc1_backward", "moe_grad_norm", "moe_grad_clip"]
    for fused in (False, True):
        for gather in (False, True):
            B.moe_layer_forward(x, wr, None, W1, W2, K, shared, bufs, fused_shared=fused, fused_route=fused,
                                gather=gather)
    assert len({n for n, _ in lib.calls}) >= 20
    for name, device in lib.calls:
        assert device == 1, name
    assert lib.real_current.current == 0
