"""The calls around the layer on tensors of a device that is not the current one (CPU only): each makes the tensors'
device current while libmoe launches, and leaves the caller's current afterwards."""

import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B
from tests.test_binding_device import E, FakeTensor, H, I, I_S, K, T, fill, lib  # noqa: F401  (lib: a fixture)

F32 = torch.float32


@pytest.mark.parametrize("layout", [B.MOE_W_KN, B.MOE_W_NK])
def test_block_calls_launch_on_the_tensors_device(lib, monkeypatch, layout):  # noqa: F811
    nk = layout == B.MOE_W_NK
    h, wr, d_out, w = FakeTensor(T, H), FakeTensor(H, E), FakeTensor(T, H), FakeTensor(H)
    W1 = FakeTensor(E, 2 * I, H) if nk else FakeTensor(E, H, 2 * I)
    W2 = FakeTensor(E, H, I) if nk else FakeTensor(E, I, H)
    shared = ((FakeTensor(2 * I_S, H), FakeTensor(H, I_S)) if nk else (FakeTensor(H, 2 * I_S), FakeTensor(I_S, H)))
    shared += (FakeTensor(H),)
    device = h.device
    with monkeypatch.context() as m:
        for name in ("empty", "zeros"):
            m.setattr(torch, name, lambda shape, dtype=None, device=None: FakeTensor(*shape, dtype=dtype))
        bufs = B.MoELayerBuffers(T, H, E, K, I, I_S, torch.bfloat16, device)
        train = B.MoETrainBuffers(T, H, E, K, I, I_S, True, False, torch.bfloat16, device, layout)
        block = B.MoEBlockBuffers(T, H, E, torch.bfloat16, torch.bfloat16, device, True, True)
        state = B.MoEOrthogonalState(wr, W1, W2, shared, layout)
        monkeypatch.setattr(FakeTensor, "view", lambda self, shape: FakeTensor(*shape, dtype=self.dtype), raising=False)
        B.moe_block_train_forward(h, w, w, w, wr, None, W1, W2, K, shared, bufs, train, block, layout=layout)
        B.moe_block_backward(d_out, h, w, w, w, wr, W1, W2, shared, bufs, train, block, max_norm=1.0, layout=layout)
        B.moe_layer_orthogonal_step(wr, W1, W2, shared, train, state, 0.1)
    names = [n for n, _ in lib.calls]
    assert names == ["moe_norm_residual", "moe_route", "moe_build_scatter", "moe_grouped_swiglu_fc1_save",
                     "moe_grouped_fc2", "moe_gather_combine", "moe_shared_fc1_save", "moe_shared_fc2_save",
                     "moe_balance_loss", "moe_norm_residual", "moe_norm_residual_backward", "moe_scatter_grad",
                     "moe_grouped_fc2_backward", "moe_grouped_fc1_backward", "moe_route_balance_backward",
                     "moe_shared_fc2_backward", "moe_shared_fc1_backward", "moe_norm_residual_backward",
                     "moe_grad_norm", "moe_grad_clip"] + ["moe_orthogonal_update"] * 5
    for name, current in lib.calls:
        assert current == 1, name
    assert lib.real_current.current == 0
