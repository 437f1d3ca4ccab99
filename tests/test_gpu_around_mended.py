"""Calls around the layer where they once went wrong, against float64."""

import numpy as np
import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B
from oracle import around_oracle as O
from tests.test_gpu_around import (COEFS, DEV, TYPES, U, balance_call, check_route, gen, half, host, normal, ortho_call,
                                   route_call, route_state, within)
from tests.test_gpu_around_large import STORE, fro, steps64
from tests.test_gpu_block import F32, KW, block_case

pytestmark = pytest.mark.gpu
BACK = {n: v for n, v in KW.items() if n != "eps"}


# ------------------------------------------------------------------------------------------
# clipping
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("name", ["d_w1", "d_w2", "d_w_router"])
def test_a_layer_gradient_replaced_between_steps_is_clipped(name):
    """The norm and the clipping take the tensors that the layer's buffers hold in that call."""
    T, H, E, k, I = 33, 64, 4, 2, 24
    p = block_case(T, H, E, k, I, 0, F32, 61, True, True, False, False, B.MOE_W_KN)
    bufs = B.MoELayerBuffers(T, H, E, k, I, 0, F32, DEV)
    train = B.MoETrainBuffers(T, H, E, k, I, 0, False, False, F32, DEV)
    block = B.MoEBlockBuffers(T, H, E, F32, F32, DEV, True, True)
    d_out = normal(gen(62), (T, H))

    def block_step(max_norm):
        B.moe_block_train_forward(p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], None, p["W1"], p["W2"], k,
                                  None, bufs, train, block, **KW)
        B.moe_block_backward(d_out, p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], p["W1"], p["W2"], None,
                             bufs, train, block, max_norm=max_norm, **BACK)
        return [host(g) for g in (train.d_w1, train.d_w2, train.d_w_router, block.d_w_pre, block.d_w_post, block.d_gate)]

    def layer_step(max_norm):
        B.moe_layer_train_forward(p["h"], p["w_router"], None, p["W1"], p["W2"], k, None, bufs, train)
        B.moe_layer_backward(d_out, p["h"], p["w_router"], p["W1"], p["W2"], None, bufs, train, max_norm)
        return [host(g) for g in (train.d_w1, train.d_w2, train.d_w_router)]

    for step, norm in ((block_step, lambda: block.norm), (layer_step, lambda: train.norm)):
        raw = step(None)
        total = sum(float((g ** 2).sum()) for g in raw) ** 0.5
        step(0.5 * total)
        setattr(train, name, torch.zeros_like(getattr(train, name)))
        for got, want in zip(step(0.25 * total), raw):
            # the same gradients times a factor: two roundings of it, one of the product
            assert np.abs(got - 0.25 * want).max() <= 1e-5 * np.abs(want).max()
        # the squares are summed in float64; the norm is rounded once
        assert abs(norm().item() / total - 1) <= 1e-6


# ------------------------------------------------------------------------------------------
# the layer's orthogonalised step
# ------------------------------------------------------------------------------------------
def test_a_refused_step_updates_nothing():
    """One weight that is not contiguous: none of the others, nor a momentum, takes the step."""
    H, E, I = 64, 4, 24   # noqa: E741
    p = block_case(1, H, E, 2, I, 0, F32, 71, False, False, False, False, B.MOE_W_KN)
    train = B.MoETrainBuffers(8, H, E, 2, I, 0, False, False, F32, DEV)
    for g in train.grad_tensors():
        g.copy_(normal(gen(72), g.shape, 1e-3))
    state = B.MoEOrthogonalState(p["w_router"], p["W1"], p["W2"])
    strided = p["w_router"].t().contiguous().t()
    before = [p["W1"].clone(), p["W2"].clone(), strided.clone()]
    with pytest.raises(ValueError, match="w_router must be contiguous"):
        B.moe_layer_orthogonal_step(strided, p["W1"], p["W2"], None, train, state, 0.05)
    for now, was in zip((p["W1"], p["W2"], strided), before):
        assert torch.equal(now, was)
    assert not any(m.any() for m in state.momenta)


# ------------------------------------------------------------------------------------------
# router backward with the losses
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, F32])
def test_losses_alone_without_ids(dtype):
    s = route_state(200, 72, 24, 3, dtype, "some", True)
    B.moe_route_balance_backward(s["x"], s["wr"], s["logits"], s["lse"], None, None, None, s["mask"], s["counts"],
                                 s["tokens"], s["d_x"], s["d_wr"], s["d_bias"], s["rws"], 0.5, 0.1, True, top_k=3)
    check_route(s, 3, 0.5, 0.1, True, weights=False)


@pytest.mark.parametrize("T,E,far", [(130, 60, 3e3), (65, 8, 3e4), (40, 256, 3e5), (70, 12, 3e38), (8200, 10, 3e4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, F32])
def test_logits_far_from_zero(T, E, far, dtype):
    """Rows of logits far from zero, the lowest ones of the type among them: lse's half step is then no small part of
    1, and probabilities taken as exp(logits - lse) alone would all be off by that factor (all equal: by E).  The
    reference takes the softmax of the logits itself.  exp is within 2 ulp of an argument that is exact next to the
    maximum (both are multiples of the same step) and rounded to |argument| U elsewhere, where p <= exp(argument):
    below 8 U of 1 in all; then the sums over E and the products."""
    k, H, coef = 2, 40, 0.7
    s = route_state(T, H, E, k, dtype, "some", True, seed=T)
    s["logits"] += far * torch.where(torch.arange(T, device=DEV) % 2 == 0, 1.0, -1.0)[:, None]
    s["logits"].clamp_(-3e38, 3e38)
    s["logits"][3] = -far
    balance_call(s)
    s["dw"].zero_()
    route_call(s, coef, 0.0, False)
    p = torch.softmax(s["logits"].double(), 1) * (s["mask"][:, None])
    c, n = s["counts"].double(), max(int(s["tokens"]), 1)
    f = coef * E / (k * n * n)
    d = p * f * (c - (p * c).sum(1, keepdim=True))
    mag = p * f * (c + (p * c).sum(1, keepdim=True))
    err = (4 * E + 48) * U * mag
    within(s["d_bias"], host(d.sum(0)), host(err.sum(0) + (T + 16) * U * mag.sum(0)), "d_logit_bias")
    wr = s["wr"].double().abs().t().contiguous()
    left = 2.0 ** -24 if dtype == torch.bfloat16 else 0.0
    within(s["d_x"], host(d @ s["wr"].double().t().contiguous()),
           host((err + (left + (3 * E + 16) * U) * (mag + err)) @ wr), "d_x")
    x = s["x"].double().abs().t().contiguous()
    left = 2.0 ** -16 if dtype == torch.bfloat16 else 0.0
    want = s["x"].double().t().contiguous() @ d
    within(s["d_wr"], host(want), host(half(dtype) * want.abs() + (1 + half(dtype))
                                       * (x @ (err + (left + (2 * T + 32) * U) * (mag + err)))), "d_w_router")


# ------------------------------------------------------------------------------------------
# orthogonalised update of few rows
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("M,N", [(2, 64), (64, 2), (4, 40), (7, 50), (8, 104), (2048, 8), (16, 64), (24, 200), (30, 300),
                                 (32, 4096)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("momentum", [False, True])
def test_few_rows_with_one_strong_direction(M, N, dt, momentum):
    """Nearly one direction, the others 1 to 1e5 times smaller: their squared singular values, which the steps on the
    Gram matrix work on, are lost first.  Beside the result's own rounding to bf16 (root mean square 0.735 / sqrt(3)
    2^-8 over mantissas whose logarithms are uniform; a quarter more for the 128 elements of the smallest) are left:
    Q, up to 490, in float32, and its float32 sums of up to 32 terms times X: sqrt(32) 490 2^-25 = 0.8e-4.  With a
    momentum the update is a float32 of its own, g + mu m rounded once: a half step of the strong direction is no small
    part of the others, so the reference starts from that float32."""
    batch = 8
    g = gen(M + N)
    for noise in [10.0 ** (-e / 4) for e in range(21)]:
        u = normal(g, (batch, M, 1)) * normal(g, (batch, 1, N)) + noise * normal(g, (batch, M, N))
        grad = u.to(TYPES[dt])
        mom = normal(g, grad.shape, 0.1 * noise) if momentum else None
        out = torch.full(grad.shape, 9.0, dtype=torch.bfloat16, device=DEV)
        ortho_call(grad, out, mom)
        u = grad.double() if mom is None else (grad.double() + float(np.float32(0.95)) * mom.double()).float()
        for i in range(batch):
            want = steps64(u[i], COEFS)
            err = fro(out[i] - want) / fro(want)
            assert err <= 1.25 * STORE + 3e-4, (noise, i)


# ------------------------------------------------------------------------------------------
# float32 weights beside bf16 gradients, and a bf16 stream
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("layout", [B.MOE_W_KN, B.MOE_W_NK])
def test_small_steps_of_float32_weights_add_up(layout):
    """Steps that a bf16 weight would lose, on float32 weights with the layer's bf16 gradients."""
    H, E, I, I_s = 96, 12, 40, 56   # noqa: E741
    p = block_case(1, H, E, 2, I, I_s, torch.bfloat16, 81, False, False, False, False, layout)
    names = ("w_router", "W1", "W2", "ws1", "ws2")
    train = B.MoETrainBuffers(8, H, E, 2, I, I_s, False, False, torch.bfloat16, DEV, layout)
    grads = dict(zip(names, (train.d_w_router, train.d_w1, train.d_w2, train.d_ws1, train.d_ws2)))
    masters = {n: p[n].float() for n in names}
    give = lambda: (masters["w_router"], masters["W1"], masters["W2"], (masters["ws1"], masters["ws2"], None))   # noqa: E731
    state = B.MoEOrthogonalState(*give(), layout)
    lr, decay = 1e-5, 0.1
    weights, moments = {n: host(m) for n, m in masters.items()}, {n: np.zeros(m.shape) for n, m in masters.items()}
    for t in range(3):
        for v in grads.values():
            v.copy_(normal(gen(82 + t), v.shape, 1e-3))
        B.moe_layer_orthogonal_step(*give(), train, state, lr, weight_decay=decay)
        for n, v in grads.items():
            a, m, w = (x if x.ndim == 3 else x[None] for x in (host(v), moments[n], weights[n]))
            parts, fused = 1, n in ("W1", "ws1")
            if fused and layout == B.MOE_W_KN:
                parts = 2
            elif fused:
                a, m, w = (x.reshape(2 * x.shape[0], x.shape[1] // 2, x.shape[2]) for x in (a, m, w))
            scale = -lr * 0.2 * max(a.shape[1], a.shape[2] // parts) ** 0.5
            w, m = O.orthogonal_update(a, w, m, 0.95, True, parts, COEFS, 1e-7, scale, 1 - lr * decay)
            weights[n], moments[n] = w.reshape(v.shape), m.reshape(v.shape)
    for n in names:
        moved = np.linalg.norm(weights[n] - host(p[n]))
        # a fused multiply-add per step and the factors' own half steps (of keep and of scale); the update itself is
        # off by a few 1e-6 of what it moves
        bound = 3 * 2 * U * np.linalg.norm(weights[n]) + 1e-5 * moved
        assert np.linalg.norm(host(masters[n]) - weights[n]) <= bound < 0.2 * moved, n
    bf16 = {n: p[n].clone() for n in names}
    for n in names:
        bf16[n].copy_(masters[n])
        assert (host(bf16[n]) == host(p[n])).mean() > 0.5, n   # most are still where they were


@pytest.mark.parametrize("rs", [1.0, 0.9])
def test_stream_gradient_of_a_bf16_block(rs):
    """d_h = rs d_h_out + the first norm's part, of what the layer's backward left: its own half step, and one of the
    first term where rs is not 1."""
    T, H, E, k, I = 50, 136, 4, 2, 24   # noqa: E741
    p = block_case(T, H, E, k, I, 0, torch.bfloat16, 91, True, True, False, False, B.MOE_W_KN)
    bf = torch.bfloat16
    bufs, train = B.MoELayerBuffers(T, H, E, k, I, 0, bf, DEV), B.MoETrainBuffers(T, H, E, k, I, 0, False, False, bf, DEV)
    block = B.MoEBlockBuffers(T, H, E, bf, bf, DEV, True, True)
    d_out = normal(gen(92), (T, H), 1.0, bf)
    kw = KW | dict(residual_scale=rs)
    B.moe_block_train_forward(p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], None, p["W1"], p["W2"], k, None,
                              bufs, train, block, **kw)
    B.moe_block_backward(d_out, p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], p["W1"], p["W2"], None, bufs,
                         train, block, **{n: v for n, v in kw.items() if n != "eps"})
    part, _ = O.norm_backward(host(train.d_x), host(p["h"]), host(block.rstd_pre), host(p["w_pre"]), KW["weight_offset"])
    want = rs * host(d_out) + part
    half_bf, mag = 2.0 ** -8, np.abs(host(d_out)) + np.abs(part)
    bound = half_bf * (np.abs(want) + (np.abs(rs * host(d_out)) if rs != 1.0 else 0.0)) * (1 + half_bf) \
        + (2 * H + 64) * U * (mag + np.abs(part).max())
    within(block.d_h, want, bound, "d_h")


# ------------------------------------------------------------------------------------------
# a whole step of a block, as a program runs it
# ------------------------------------------------------------------------------------------
class Step:
    """Forward, backward with clipping, and the update of the layer's weights."""

    def __init__(self, seed, T=130, H=136, E=6, k=2, I=40, I_s=48, dtype=torch.bfloat16):  # noqa: E741
        self.p = p = block_case(T, H, E, k, I, I_s, dtype, seed, True, True, True, True, B.MOE_W_KN)
        self.k, self.shared = k, (p["ws1"], p["ws2"], p["w_gate"])
        self.bufs = B.MoELayerBuffers(T, H, E, k, I, I_s, dtype, DEV)
        self.train = B.MoETrainBuffers(T, H, E, k, I, I_s, True, True, dtype, DEV)
        self.block = B.MoEBlockBuffers(T, H, E, dtype, dtype, DEV, True, True)
        self.state = B.MoEOrthogonalState(p["w_router"], p["W1"], p["W2"], self.shared)
        self.mask = torch.rand((T,), generator=gen(seed + 1), device=DEV) < 0.8
        self.d_out = normal(gen(seed + 2), (T, H), 1.0, dtype)

    def run(self, stream=None):
        p, layer = self.p, (self.shared, self.bufs, self.train)
        B.moe_block_train_forward(p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], p["bias"], p["W1"], p["W2"],
                                  self.k, *layer, self.block, self.mask, stream=stream, **KW)
        B.moe_block_backward(self.d_out, p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], p["W1"], p["W2"],
                             *layer, self.block, self.mask, max_norm=0.5, stream=stream, **BACK)
        B.moe_layer_orthogonal_step(p["w_router"], p["W1"], p["W2"], self.shared, self.train, self.state, 0.02,
                                    weight_decay=0.1, stream=stream)

    def out(self):
        b, t, p = self.block, self.train, self.p
        return [b.h_out, b.losses, b.counts, b.d_h, b.d_w_pre, b.d_w_post, b.d_gate, b.norm, *t.grad_tensors(), t.d_x,
                p["W1"], p["W2"], p["w_router"], p["ws1"], p["ws2"], *self.state.momenta]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a.out(), b.out()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, F32])
def test_whole_step_captured_and_replayed(dtype):
    """Each replay takes one more step; the program's own work lies between them."""
    eager, c, other = Step(101, dtype=dtype), Step(101, dtype=dtype), Step(102, dtype=dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(side)
    torch.cuda.current_stream().wait_stream(side)
    eager.run()
    assert same(eager, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(4):
        graph.replay()
        other.run()
        torch.cuda.synchronize()
        eager.run()
        assert same(eager, c)


def test_two_whole_steps_at_once():
    a, b, want_a, want_b = (Step(s) for s in (103, 104, 103, 104))
    for _ in range(3):
        want_a.run()
        want_b.run()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, x in zip(streams, (a, b)):
            x.run(s)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert same(a, want_a) and same(b, want_b)
