"""A training step of the block around the layer, and the calls around the layer as a program uses them: captured and
replayed, on other streams, two at once, repeated."""

import numpy as np
import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B
from oracle import around_oracle as O
from tests.test_gpu_around import (COEFS, DEV, EVERY, QUINTIC, balance_call, gen, host, matrices, norm_backward,
                                   norm_forward, norm_state, normal, ortho_bound, ortho_call, rel, route_call,
                                   route_state, ws)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------------------------
# every call as one object: its inputs, its run, its outputs
# ------------------------------------------------------------------------------------------
class Balance:
    def __init__(self, seed):
        self.s = route_state(333, 128, 60, 4, BF16, "some", True, seed)

    def run(self, stream=None):
        balance_call(self.s, stream=stream)
        self.s["d_x"].copy_(self.s["old"]) if stream is None else None
        route_call(self.s, 0.3, 0.2, False, stream=stream)

    def out(self):
        return [self.s[n] for n in ("losses", "counts", "tokens", "prob_sums", "lse", "d_x", "d_wr", "d_bias")]


class Norm:
    def __init__(self, seed):
        self.s = norm_state(300, 1032, BF16, BF16, **EVERY, seed=seed)

    def run(self, stream=None):
        norm_forward(self.s, stream)
        norm_backward(self.s, stream)

    def out(self):
        return [self.s[n] for n in ("h_out", "x", "rstd_post", "rstd_pre", "d_h", "d_y", "d_w_pre", "d_w_post", "d_gate")]


class Ortho:
    def __init__(self, seed, M, N, dtype=BF16, batch=2):
        g = gen(seed)
        self.grad = matrices(g, (batch, M, N), "strong", dtype)
        self.w, self.m = normal(g, self.grad.shape, 0.1, dtype), normal(g, self.grad.shape, 1e-3)
        self.ws = ws(B.moe_orthogonal_update_workspace_bytes(dtype, dtype, batch, M, N, 1, True))

    def run(self, stream=None):   # in place: every run is another step
        ortho_call(self.grad, self.w, self.m, workspace=self.ws, stream=stream, scale=-0.1, keep=0.9)

    def out(self):
        return [self.w, self.m]


CALLS = {"balance": Balance, "norm": Norm, "ortho_narrow": lambda seed: Ortho(seed, 60, 300),
         "ortho_gram": lambda seed: Ortho(seed, 1000, 140), "ortho": lambda seed: Ortho(seed, 264, 320),
         "ortho_f32": lambda seed: Ortho(seed, 96, 140, F32)}


def copies(outs):
    return [o.clone() for o in outs]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", CALLS)
def test_same_bits_again_and_whatever_the_workspace_held(name):
    first, second = CALLS[name](1), CALLS[name](1)
    first.run()
    for key in ("ws", "rws"):
        held = second.__dict__.get(key) if key in second.__dict__ else getattr(second, "s", {}).get(key)
        if held is not None:
            held.fill_(0xFF)
    second.run()
    assert same(first.out(), second.out())


@pytest.mark.parametrize("name", CALLS)
def test_captured_and_replayed(name):
    eager, c = CALLS[name](2), CALLS[name](2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(side)                    # a warm-up run; in-place updates take a step on both sides
    torch.cuda.current_stream().wait_stream(side)
    eager.run(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(torch.cuda.current_stream())
    other = CALLS[name](3)
    for _ in range(3):
        graph.replay()
        other.run()                    # the program's own work between replays
        torch.cuda.synchronize()
        eager.run(torch.cuda.current_stream())
        assert same(eager.out(), c.out())


@pytest.mark.parametrize("name", CALLS)
def test_two_at_once_on_two_streams(name):
    a, b, want_a, want_b = (CALLS[name](i) for i in (4, 5, 4, 5))
    for _ in range(3):
        want_a.run(torch.cuda.current_stream())
        want_b.run(torch.cuda.current_stream())
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.run(s1)
        b.run(s2)
    for s in (s1, s2):
        torch.cuda.current_stream().wait_stream(s)
    assert same(a.out(), want_a.out()) and same(b.out(), want_b.out())


def test_a_stack_is_its_matrices():
    """A matrix's result does not depend on what it is stacked with (up to the tiles that the stack's size picks)."""
    for M, N in ((40, 90), (150, 170), (140, 900)):
        grad = matrices(gen(8), (5, M, N), "strong", BF16)
        out, one = torch.zeros_like(grad), torch.zeros((1, M, N), dtype=BF16, device=DEV)
        ortho_call(grad, out)
        for i in (0, 4):
            ortho_call(grad[i:i + 1].contiguous(), one)
            assert rel(one[0], host(out[i])) <= 2 * ortho_bound(BF16, N)


def test_many_matrices_and_long_ones():
    """Stacks that fill the chip take the large tiles; sides that end inside them."""
    for shape in ((40, 520, 700), (3, 1300, 1100), (2, 136, 5000), (300, 24, 40), (1, 2600, 2700)):
        grad = matrices(gen(sum(shape)), shape, "strong", BF16)
        out = torch.zeros_like(grad)
        ortho_call(grad, out)
        for i in {0, shape[0] - 1}:
            x = grad[i].double()
            x = x / (x.norm() + 1e-7)
            for a, b, c in COEFS:
                gram = x @ x.t().contiguous()
                x = a * x + (b * gram + c * gram @ gram) @ x
            assert rel(out[i], host(x)) <= ortho_bound(BF16, max(shape[1:])), shape


def test_more_than_32_bits_of_elements():
    """A stack of more than 2^32 bytes per tensor: its last matrix as by itself."""
    shape = (9000, 512, 500)
    g = gen(11)
    grad = torch.empty(shape, dtype=BF16, device=DEV)
    for i in range(0, shape[0], 1000):
        grad[i:i + 1000] = matrices(g, (1000, *shape[1:]), "noise", BF16)
    out = torch.zeros_like(grad)
    ortho_call(grad, out)
    one = torch.zeros((1, *shape[1:]), dtype=BF16, device=DEV)
    for i in (0, 8999):
        ortho_call(grad[i:i + 1].contiguous(), one)
        assert rel(one[0], host(out[i])) <= 2 * ortho_bound(BF16, 512)


def test_norm_of_more_than_32_bits_of_elements():
    T, H = 600_000, 8192
    h = torch.empty((T, H), dtype=BF16, device=DEV)
    h[:1000] = normal(gen(12), (1000, H), 1.0, BF16)
    h[-1000:] = h[:1000]
    w = normal(gen(13), (H,), 0.5, BF16)
    x, r = torch.empty_like(h), torch.empty((T,), device=DEV)
    B.moe_norm_residual(h, None, None, None, w, None, x, None, r)
    assert torch.equal(x[:1000], x[-1000:]) and torch.equal(r[:1000], r[-1000:])
    want, _ = O.norm(host(h[:4]), host(w))
    assert rel(x[:4], want) <= 2.0 ** -8


# ------------------------------------------------------------------------------------------
# the block
# ------------------------------------------------------------------------------------------
def block_reference(p, ids, counts, mask, top_k, kw):
    """(h_out, losses) of the block in torch float64 on the CPU, routes held fixed; p: name -> tensor or None."""
    def norm(v, w):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + kw["eps"]) * (kw["weight_offset"] + w)

    x = norm(p["h"], p["w_pre"])
    logits = x @ p["w_router"] + (0 if p["bias"] is None else p["bias"])
    q = torch.softmax(logits.gather(1, ids), 1)
    T, E = logits.shape
    y = torch.zeros_like(x)
    for e in range(E):
        for j in range(top_k):
            rows = (ids[:, j] == e).nonzero()[:, 0]
            if len(rows):
                g, u = (x[rows] @ p["W1"][e]).chunk(2, 1)
                y = y.index_add(0, rows, q[rows, j:j + 1] * ((torch.nn.functional.silu(g) * u) @ p["W2"][e]))
    if p["ws1"] is not None:
        g, u = (x @ p["ws1"]).chunk(2, 1)
        ys = (torch.nn.functional.silu(g) * u) @ p["ws2"]
        y = y + (torch.sigmoid(x @ p["w_gate"])[:, None] * ys if p["w_gate"] is not None else ys)
    n = y if p["w_post"] is None else norm(y, p["w_post"])
    n = n if p["gate"] is None else n * p["gate"]
    h_out = kw["residual_scale"] * p["h"] + kw["branch_scale"] * n
    valid = torch.ones(T, dtype=torch.float64) if mask is None else mask.double()
    nv = valid.sum().clamp(min=1)
    lse = torch.logsumexp(logits, 1)
    probs = torch.softmax(logits, 1)
    balance = kw["balance_coef"] * E / (top_k * nv * nv) * (counts * (probs * valid[:, None]).sum(0)).sum()
    return h_out, torch.stack([balance, kw["z_coef"] / nv * (valid * lse * lse).sum()])


def block_case(T, H, E, k, I, I_s, dtype, seed, post, gate, gated, bias, layout):
    g = gen(seed)
    nk = layout == B.MOE_W_NK
    w = lambda *shape: normal(g, shape, 0.5 / shape[-1 if nk else -2] ** 0.5, dtype)   # noqa: E731
    p = {"h": normal(g, (T, H), 1.0, dtype), "w_pre": normal(g, (H,), 0.2, dtype),
         "w_post": normal(g, (H,), 0.2, dtype) if post else None,
         "gate": normal(g, (H,), 0.5, dtype) if gate else None, "w_router": normal(g, (H, E), 0.3, dtype),
         "bias": normal(g, (E,), 0.1) if bias else None,
         "W1": w(E, 2 * I, H) if nk else w(E, H, 2 * I), "W2": w(E, H, I) if nk else w(E, I, H),
         "ws1": None, "ws2": None, "w_gate": None}
    if I_s:
        p |= {"ws1": w(2 * I_s, H) if nk else w(H, 2 * I_s), "ws2": w(H, I_s) if nk else w(I_s, H),
              "w_gate": normal(g, (H,), 0.2, dtype) if gated else None}
    return p


KW = dict(balance_coef=0.5, z_coef=0.2, eps=1e-5, weight_offset=1.0, residual_scale=0.9, branch_scale=0.6)


@pytest.mark.parametrize("layout", [B.MOE_W_KN, B.MOE_W_NK])
@pytest.mark.parametrize("post,gate,I_s,gated,bias,masked", [
    (True, True, 48, True, True, True), (False, False, 0, False, False, False), (True, False, 40, False, True, False),
    (False, True, 48, True, False, True)])
def test_block_step_against_autograd(layout, post, gate, I_s, gated, bias, masked):
    """Loss, stream and every gradient of a float32 block against torch's autograd in float64, and a clipped step's
    norm; float32 products of up to 256 terms: the layer's own bound of 1e-4."""
    T, H, E, k, I = 61, 72, 6, 2, 40
    p = block_case(T, H, E, k, I, I_s, F32, 21, post, gate, gated, bias, layout)
    shared = None if not I_s else (p["ws1"], p["ws2"], p["w_gate"])
    bufs = B.MoELayerBuffers(T, H, E, k, I, I_s, F32, DEV)
    train = B.MoETrainBuffers(T, H, E, k, I, I_s, gated, bias, F32, DEV, layout)
    block = B.MoEBlockBuffers(T, H, E, F32, F32, DEV, post, gate)
    mask = torch.rand((T,), generator=gen(22), device=DEV) < 0.8 if masked else None
    d_out = normal(gen(23), (T, H))
    B.moe_block_train_forward(p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], p["bias"], p["W1"], p["W2"], k,
                              shared, bufs, train, block, mask, layout=layout, **KW)
    back = {n: v for n, v in KW.items() if n != "eps"}
    args = (d_out, p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], p["W1"], p["W2"], shared, bufs, train,
            block, mask)
    B.moe_block_backward(*args, layout=layout, **back)

    nk = layout == B.MOE_W_NK
    ref = {n: None if v is None else v.detach().double().cpu() for n, v in p.items()}
    leaves = {n: v.requires_grad_() for n, v in ref.items() if v is not None}
    used = {n: v.transpose(-1, -2) if nk and n in ("W1", "W2", "ws1", "ws2") and v is not None else v
            for n, v in ref.items()}
    h_out, losses = block_reference(used, bufs.topk_ids.cpu().long(), block.counts.cpu().double(),
                                    None if mask is None else mask.cpu(), k, KW)
    ((h_out * d_out.double().cpu()).sum() + losses.sum()).backward()
    assert rel(block.h_out, h_out.detach().numpy()) <= 1e-5 and rel(block.losses, losses.detach().numpy()) <= 1e-5
    got = {"h": block.d_h, "w_pre": block.d_w_pre, "w_post": block.d_w_post, "gate": block.d_gate,
           "w_router": train.d_w_router, "bias": train.d_logit_bias, "W1": train.d_w1, "W2": train.d_w2,
           "ws1": train.d_ws1, "ws2": train.d_ws2, "w_gate": train.d_w_gate}
    total = 0.0
    for n, leaf in leaves.items():
        assert rel(got[n], leaf.grad.numpy()) <= 1e-4, n
        total += 0.0 if n == "h" else float((leaf.grad ** 2).sum())
    B.moe_block_backward(*args, layout=layout, max_norm=0.5 * total ** 0.5, **back)
    assert abs(block.norm.item() / total ** 0.5 - 1) <= 1e-4 and abs(block.coef.item() - 0.5) <= 1e-4
    assert rel(train.d_w1, 0.5 * leaves["W1"].grad.numpy()) <= 3e-4


@pytest.mark.parametrize("layout", [B.MOE_W_KN, B.MOE_W_NK])
def test_orthogonal_step_of_a_layer(layout):
    T, H, E, k, I, I_s = 100, 96, 5, 2, 40, 56
    p = block_case(T, H, E, k, I, I_s, BF16, 31, True, True, True, True, layout)
    shared = (p["ws1"], p["ws2"], p["w_gate"])
    train = B.MoETrainBuffers(T, H, E, k, I, I_s, True, True, BF16, DEV, layout)
    g = gen(32)
    grads = {"W1": train.d_w1, "W2": train.d_w2, "w_router": train.d_w_router, "ws1": train.d_ws1, "ws2": train.d_ws2}
    state = B.MoEOrthogonalState(p["w_router"], p["W1"], p["W2"], shared, layout)
    weights = {n: host(p[n]) for n in grads}
    moments = {n: np.zeros(p[n].shape) for n in grads}
    for _ in range(2):
        for v in grads.values():
            v.copy_(normal(g, v.shape, 1e-3))
        B.moe_layer_orthogonal_step(p["w_router"], p["W1"], p["W2"], shared, train, state, 0.05, weight_decay=0.1)
        for n, v in grads.items():
            a, m, w = (x if x.ndim == 3 else x[None] for x in (host(v), moments[n], weights[n]))
            parts = 1
            if n in ("W1", "ws1") and layout == B.MOE_W_KN:
                parts = 2
            elif n in ("W1", "ws1"):
                a, m, w = (x.reshape(2 * x.shape[0], x.shape[1] // 2, x.shape[2]) for x in (a, m, w))
            scale = -0.05 * 0.2 * max(a.shape[1], a.shape[2] // parts) ** 0.5
            w, m = O.orthogonal_update(a, w, m, 0.95, True, parts, COEFS, 1e-7, scale, 1 - 0.05 * 0.1)
            # the weight's own rounding in each of two steps, and the update's error
            step = np.linalg.norm(scale * np.ones(a.shape)) / max(a.shape[1], a.shape[2]) ** 0.5
            err = np.linalg.norm(host(p[n]).reshape(w.shape) - w)
            assert err <= 2 * (2.0 ** -8 * np.linalg.norm(w) + ortho_bound(BF16, 96) * step), n
            weights[n], moments[n] = host(p[n]), m.reshape(p[n].shape)
    with pytest.raises(ValueError, match="without a shared expert|with a shared expert"):
        B.moe_layer_orthogonal_step(p["w_router"], p["W1"], p["W2"], None, train, state, 0.05)
    assert QUINTIC == B.ORTHOGONAL_COEFS[0]


def test_block_of_one_token_and_bf16_stream():
    """Decode's sizes: one token through both norms and the layer, bf16 throughout, finite and near float64."""
    T, H, E, k, I = 1, 128, 4, 2, 64
    p = block_case(T, H, E, k, I, 0, BF16, 41, True, True, False, False, B.MOE_W_KN)
    bufs = B.MoELayerBuffers(T, H, E, k, I, 0, BF16, DEV)
    train = B.MoETrainBuffers(T, H, E, k, I, 0, False, False, BF16, DEV)
    block = B.MoEBlockBuffers(T, H, E, BF16, BF16, DEV, True, True)
    B.moe_block_train_forward(p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], None, p["W1"], p["W2"], k, None,
                              bufs, train, block, **KW)
    B.moe_block_backward(normal(gen(42), (T, H), 1.0, BF16), p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"],
                         p["W1"], p["W2"], None, bufs, train, block,
                         **{n: v for n, v in KW.items() if n != "eps"})
    ref = {n: None if v is None else v.double().cpu() for n, v in p.items()}
    h_out, losses = block_reference(ref, bufs.topk_ids.cpu().long(), block.counts.cpu().double(), None, k, KW)
    # x, act and the stream are stored in bf16 on the way: a few half steps
    assert rel(block.h_out, h_out.numpy()) <= 4 * 2.0 ** -8 and rel(block.losses, losses.numpy()) <= 4 * 2.0 ** -8
    for g in (block.d_h, block.d_w_pre, block.d_w_post, block.d_gate, train.d_w1, train.d_w_router):
        assert torch.isfinite(g.float()).all()


def test_block_gradients_replaced_between_steps():
    """A step clips the gradients that the buffers hold now, whatever they and ``train`` were in the step before."""
    T, H, E, k, I = 33, 64, 4, 2, 24
    p = block_case(T, H, E, k, I, 0, F32, 51, True, True, False, False, B.MOE_W_KN)
    bufs = B.MoELayerBuffers(T, H, E, k, I, 0, F32, DEV)
    block = B.MoEBlockBuffers(T, H, E, F32, F32, DEV, True, True)
    d_out = normal(gen(52), (T, H))
    back = {n: v for n, v in KW.items() if n != "eps"}

    def step(train, max_norm):
        B.moe_block_train_forward(p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], None, p["W1"], p["W2"], k,
                                  None, bufs, train, block, **KW)
        B.moe_block_backward(d_out, p["h"], p["w_pre"], p["w_post"], p["gate"], p["w_router"], p["W1"], p["W2"], None,
                             bufs, train, block, max_norm=max_norm, **back)
        return [host(g) for g in (train.d_w1, train.d_w2, train.d_w_router, block.d_w_pre, block.d_w_post, block.d_gate)]

    first, second = (B.MoETrainBuffers(T, H, E, k, I, 0, False, False, F32, DEV) for _ in range(2))
    raw = step(first, None)
    total = sum(float((g ** 2).sum()) for g in raw) ** 0.5
    step(first, 0.5 * total)
    block.d_gate, block.d_w_pre = torch.empty_like(block.d_gate), torch.empty_like(block.d_w_pre)
    for got, want in zip(step(second, 0.25 * total), raw):
        # the same gradients times a factor: two roundings of it, one of the product
        assert np.abs(got - 0.25 * want).max() <= 1e-5 * np.abs(want).max()
    # the squares are summed in float64; the norm is rounded once
    assert abs(block.norm.item() / total - 1) <= 1e-6
