"""The binding's calls around the layer: what they take from the buffers, and what they refuse (CPU only)."""

import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B
from tests.test_binding_device import E, FakeTensor, H, I, I_S, K, T, fill, lib  # noqa: F401  (lib: a fixture)

NAMES = ("d_w1", "d_w2", "d_w_router", "d_logit_bias", "d_ws1", "d_ws2", "d_w_gate")


def test_gradient_lists_hold_what_the_buffers_hold_now(lib, monkeypatch):  # noqa: F811
    train = fill(monkeypatch, B.MoETrainBuffers, T, H, E, K, I, I_S, True, True)
    block = fill(monkeypatch, lambda *a: B.MoEBlockBuffers(T, H, E, a[0], a[0], a[1], True, True))
    for name in NAMES:
        new = FakeTensor(*getattr(train, name).shape)
        setattr(train, name, new)
        now = [getattr(train, n) for n in NAMES]
        assert [id(g) for g in train.grads.grads] == [id(g) for g in now], name
        now += [block.d_w_pre, block.d_w_post, block.d_gate]
        assert [id(g) for g in block.grad_list(train).grads] == [id(g) for g in now], name
