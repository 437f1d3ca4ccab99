"""The calls around the layer at sizes that take every kind of launch, against float64 with bounds near what is
documented of them."""

import math

import numpy as np
import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B
from oracle import around_oracle as O
from tests.test_gpu_around import (COEFS, DEV, QUINTIC, TYPES, U, balance_call, balance_state, gen, host, matrices,
                                   normal, ortho_call, within)

pytestmark = pytest.mark.gpu
BF16, F32, D = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------------------------------
# balance and z loss
# ------------------------------------------------------------------------------------------
def check_balance_closely(s, k, lanes):
    """Bounds by the depth of each sum.  A row: 16 values of a lane and the exchanges between its lanes; exp and log
    within 2 ulp, exp's argument rounded once (logits lie within 32 of their row's maximum).  A column: a lane's
    tokens, the groups of a wave, eight waves, 16 workgroups, 16 runs.  One token more or less in 70001 is off by
    1.4e-5 of the sums; these bounds are below 1e-5."""
    T, E = s["logits"].shape
    losses, counts, n, sums, lse = O.balance_loss(host(s["logits"]), s["ids"].cpu().numpy(), host(s["mask"]), k, 0.3, 0.2)
    assert (s["counts"].cpu().numpy() == counts).all() and int(s["tokens"]) == n
    row = (16 + math.log2(lanes) + 8 + 32) * U
    turns = -(-T // (256 * 8 * (64 // lanes) * 2)) * 2
    depth = (turns + 6 + 8 + 16 + 16) * U
    assert row + depth < 1e-5
    lse_err = row + 4 * U * np.abs(lse)
    within(s["lse"], lse, lse_err, "lse")
    within(s["prob_sums"], sums, (row + depth) * sums, "prob_sums")
    assert abs(s["prob_sums"].double().sum().item() - n) <= (row + depth) * n
    z = 0.2 / n
    within(s["losses"], losses, [(row + depth + 4 * U) * losses[0],
                                 z * float((2 * np.abs(lse) * lse_err).sum()) + (depth + 4 * U) * losses[1]], "losses")


@pytest.mark.parametrize("T,E,k,mask,lanes", [
    (140001, 16, 2, "some", 4), (90001, 30, 3, None, 4), (70001, 60, 4, "some", 4), (40001, 128, 2, None, 8),
    (40009, 127, 2, "some", 8), (32769, 256, 8, "some", 16), (32768, 256, 8, None, 16), (9001, 512, 4, "some", 32),
    (8193, 1000, 4, None, 64), (16391, 1024, 2, "some", 64), (300001, 8, 1, "some", 4)])
def test_balance_loss_of_long_batches(T, E, k, mask, lanes):
    """Two groups of tokens in flight, and up to five turns of every workgroup."""
    assert T * lanes >= 256 * 512 * 2
    s = balance_state(T, E, k, mask, seed=T + E)
    balance_call(s)
    check_balance_closely(s, k, lanes)


# ------------------------------------------------------------------------------------------
# orthogonalised update
# ------------------------------------------------------------------------------------------
# Half a step of bf16 and of fp16 (2^-8 and 2^-11 of a value in [1, 2) of its power of two), as the root mean square of
# a uniform error over mantissas whose logarithms are uniform: times 0.735 / sqrt(3).  For matrices of many elements.
STORE, HALF16 = 0.735 / 3 ** 0.5 * 2.0 ** -8, 0.735 / 3 ** 0.5 * 2.0 ** -11


def steps64(x, coefs, dtype=D):
    """The steps on X = u / (|u| + eps) in plain products of `dtype`, on the GPU."""
    x = x.to(dtype)
    tall = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if tall else x.contiguous()
    x = x / (torch.sqrt((x * x).sum()) + 1e-7)
    for a, b, c in coefs:
        gram = x @ x.t().contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.t() if tall else x


def step_of(grad, mom, nesterov=True, mu=0.95):
    """(update, momentum) in float64."""
    g = grad.double()
    if mom is None:
        return g, None
    m = mu * mom.double() + g
    return (g + mu * m if nesterov else m), m


def fro(x):
    return float(torch.linalg.vector_norm(x.double()))


def check_updates(shape, dt, odt, momentum, kind, parts=1, coefs=COEFS, keep=0.0, way="x"):
    """The first, a middle and the last matrix of a stack.

    A float32 result (and the products of many steps): operands in two fp16 parts have two bits less than float32, and
    a product leaves out that of the two low parts: at most 4 sqrt(3) < 8 times what plain float32 products are off by,
    which carry the same growth of small singular values.

    A bf16 result of steps on the Gram matrix has operands of two parts too, squared singular values: below 5e-4.  One
    of steps on X takes single fp16 operands in its products.  With s = 1 (the others are smaller where it counts): a
    step's terms b A and c A A weigh up to 2.8 of X together, so B's rounding and that of X beside it add 2.8 half
    steps each, A's own 1.4 (|b + 2 c s| s), and X's two places in A 1.4 each; sqrt(2 * 2.8^2 + 3 * 1.4^2) = 4.7 of
    them per step, independent from step to step."""
    batch, M, N = shape
    g = gen(sum(shape))
    grad = matrices(g, (batch, M, parts * N), kind, TYPES[dt])
    mom = normal(g, grad.shape, 2e-3) if momentum else None
    out = normal(g, grad.shape, 0.05, TYPES[odt])
    old, before = out.clone(), None if mom is None else mom.clone()
    ortho_call(grad, out, mom, parts, scale=-0.7, keep=keep, coefs=coefs)
    u, m = step_of(grad, before)
    if momentum:
        for i in {0, batch - 1}:
            within(mom[i], host(m[i]), host(2 * U * (m[i].abs() + grad[i].double().abs()) + 1e-12), "momentum")
    for i in sorted({0, batch // 2, batch - 1}):
        for j in range(parts):
            cols = slice(j * N, (j + 1) * N)
            x = -0.7 * steps64(u[i, :, cols], coefs)
            plain = fro(-0.7 * steps64(u[i, :, cols].float(), coefs, F32) - x)
            want = x + (keep * old[i, :, cols].double() if keep else 0.0)
            err, size = fro(out[i, :, cols] - want), fro(x)
            if odt == "f32":
                bound = 8 * plain + 2 * U * (size + fro(want))
            elif way == "deep":
                bound = 1.05 * STORE * fro(want) + 8 * plain
            elif way == "gram":
                bound = 1.05 * STORE * fro(want) + 5e-4 * size
            else:
                bound = 1.05 * math.hypot(STORE * fro(want), len(coefs) ** 0.5 * 4.7 * HALF16 * size)
            assert err <= bound, (i, j, err / size, bound / size, plain / size)


# float32 results; the tile of the symmetric products, then of those onto X
@pytest.mark.parametrize("shape,dt,momentum,parts", [
    ((24, 520, 700), "f32", False, 1),      # 128, 256
    ((40, 1000, 520), "bf16", False, 1),    # 256, 256, transposed; the first step takes X in one part
    ((40, 1000, 520), "bf16", True, 1),     # and in two
    ((8, 1024, 1024), "f32", False, 1),     # 128, 128
    ((30, 380, 250), "bf16", True, 2),      # 128, 128, transposed, side by side
    ((30, 300, 400), "f32", True, 1),       # 64, 128
    ((3, 400, 512), "bf16", True, 1),       # 64, 64
    ((2, 130, 1000), "f32", False, 1), ((16, 256, 128), "f32", False, 2), ((5, 72, 24), "bf16", True, 2)])
@pytest.mark.parametrize("kind", ["noise", "strong"])
def test_float32_results_follow_float32_products(shape, dt, momentum, parts, kind):
    check_updates(shape, dt, "f32", momentum, kind, parts)
    check_updates(shape, dt, "f32", momentum, kind, parts, keep=0.9)


@pytest.mark.parametrize("shape", [(20, 520, 700), (60, 700, 520), (60, 300, 400), (2, 150, 140)])
@pytest.mark.parametrize("momentum", [False, True])
def test_many_steps_on_every_tile(shape, momentum):
    for kind in ("noise", "strong"):
        check_updates(shape, "bf16", "bf16", momentum, kind, coefs=(QUINTIC,) * 7, way="deep")


# the tile of X0 X0^T and of the steps' products; of two of them at once; of the result
@pytest.mark.parametrize("shape,momentum", [
    ((64, 505, 2600), False), ((64, 505, 2600), True),      # 256, 128, 256
    ((250, 1301, 249), True), ((200, 136, 900), False),     # 256, 128, 128
    ((128, 250, 1300), False),                              # 128, 256, 256
    ((100, 2600, 500), True), ((40, 264, 1400), False),     # 128, 128, 256 and 128
    ((24, 264, 1400), True),                                # 64, 128, 128
    ((3, 1300, 260), True), ((1, 7168, 256), False)])       # 64, split X0 X0^T
@pytest.mark.parametrize("kind", ["noise", "strong"])
def test_long_matrices_on_every_tile(shape, momentum, kind):
    check_updates(shape, "bf16", "bf16", momentum, kind, way="gram")
    check_updates(shape, "bf16", "bf16", momentum, kind, keep=0.9, way="gram")


@pytest.mark.parametrize("shape,parts", [((40, 520, 700), 1), ((3, 1300, 1100), 1), ((2, 400, 512), 2), ((6, 1024, 1024), 1),
                                         ((2, 300, 301), 1), ((20, 700, 520), 2)])
@pytest.mark.parametrize("momentum", [False, True])
def test_steps_on_x_within_their_roundings(shape, parts, momentum):
    for kind in ("noise", "strong"):
        check_updates(shape, "bf16", "bf16", momentum, kind, parts)


# ------------------------------------------------------------------------------------------
# tensors of more than 2^31 elements: a batch of 1000 tokens again and again
# ------------------------------------------------------------------------------------------
def again(t, times):
    return None if t is None else t.repeat(times, *[1] * (t.dim() - 1))


def test_router_losses_of_more_than_32_bits_of_logits():
    """Every copy of a token gets what it gets in the batch of 1000; sums are that batch's, 2200 times."""
    times, T, E, k, H = 2200, 1000, 1000, 2, 16
    one = balance_state(T, E, k, "some", seed=5)
    big = {n: again(one[n], times) for n in ("logits", "ids", "mask", "lse")}
    assert big["logits"].numel() > 2 ** 31
    big |= {n: one[n].clone() for n in ("losses", "counts", "tokens", "prob_sums")}
    big["ws"] = torch.full((B.moe_balance_loss_workspace_bytes(T * times, E),), 0xA5, dtype=torch.uint8, device=DEV)
    balance_call(one)
    balance_call(big)
    assert torch.equal(big["counts"], times * one["counts"]) and int(big["tokens"]) == times * int(one["tokens"])
    for i in (0, times // 2, times - 1):
        assert torch.equal(big["lse"].view(times, T)[i], one["lse"])
    losses, _, n, sums, _ = O.balance_loss(host(one["logits"]), one["ids"].cpu().numpy(), host(one["mask"]), k, 0.3, 0.2)
    turns = T * times // (256 * 8)
    row, depth = (16 + 6 + 8 + 32) * U, (turns + 8 + 16 + 16) * U
    within(big["prob_sums"], times * sums, (row + depth) * times * sums, "prob_sums")
    within(big["losses"], losses, (3 * row + depth + 8 * U) * losses, "losses")   # both are means: the same

    g = gen(6)
    x, wr, old = normal(g, (T, H), 1.0, BF16), normal(g, (H, E), 0.05, BF16), normal(g, (T, H), 1e-7)
    w, dw = torch.softmax(normal(g, (T, k)), 1).contiguous(), normal(g, (T, k), 1e-7)

    def backward(s, times):
        out = [again(old, times), torch.zeros((H, E), dtype=BF16, device=DEV), torch.zeros((E,), device=DEV)]
        need = B.moe_route_balance_backward_workspace_bytes(BF16, T * times, H, E, k)
        ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV)
        B.moe_route_balance_backward(again(x, times), wr, s["logits"], s["lse"], s["ids"], again(w, times),
                                     again(dw, times), s["mask"], big["counts"], big["tokens"], *out, ws, 0.3, 0.2, True)
        return out

    d_x, d_w, d_b = backward(big, times)
    one_x, _, _ = backward(one, 1)      # with the whole batch's counts
    for i in (0, times // 2, times - 1):
        assert torch.equal(d_x.view(times, T, H)[i], one_x)
    _, want_w, want_b, d = O.route_balance_backward(host(x), host(wr), host(one["logits"]), host(one["lse"]),
                                                    one["ids"].cpu().numpy(), host(w), host(dw), host(one["mask"]),
                                                    host(big["counts"]), int(big["tokens"]), k, 0.3, 0.2)
    # d's own roundings (its terms' magnitudes are at most twice theirs without the differences), the sums by ranges
    d_err = (E + 64) * U * (np.abs(d) + 2 * np.abs(d).mean())
    full, ranges = np.abs(d) + d_err, (T * times // 16 + 32) * U
    within(d_b, times * want_b, times * (d_err.sum(0) + ranges * full.sum(0)), "d_logit_bias")
    mag = np.abs(host(x)).T
    within(d_w, times * want_w, times * (2.0 ** -8 * np.abs(want_w)
                                         + 1.01 * (mag @ d_err + (2.0 ** -16 + 2 * ranges) * (mag @ full))), "d_w_router")


def test_norm_backward_of_more_than_32_bits_of_elements():
    from tests.test_gpu_around import EVERY, check_norm_backward, norm_backward, norm_forward, norm_state
    times, T, H = 280, 1000, 8192
    assert times * T * H > 2 ** 31
    s = norm_state(T, H, BF16, BF16, **EVERY, seed=7)
    norm_forward(s)
    norm_backward(s)
    check_norm_backward(s)
    big = {n: again(s[n], times) for n in ("h", "y", "h_out", "d_h_out", "d_x", "rstd_post", "rstd_pre", "d_h", "d_y")}
    big["d_h"].fill_(9.0)
    big["d_y"].fill_(9.0)
    big |= {n: s[n] for n in ("w_post", "gate", "w_pre")}
    big |= {n: torch.zeros_like(s[n]) for n in ("d_w_pre", "d_w_post", "d_gate")}
    big["ws"] = torch.full((B.moe_norm_residual_backward_workspace_bytes(T * times, H),), 0xA5, dtype=torch.uint8,
                           device=DEV)
    norm_backward(big)
    for n in ("d_h", "d_y"):
        for i in (0, times // 2, times - 1):
            assert torch.equal(big[n].view(times, T, H)[i], s[n]), n
    # the weights' gradients: the same terms, of up to 1 per token on average (all factors are near 1 or below), in
    # sums of a workgroup's rows and 32 runs; the batch's own sums are stored within a half step
    for n in ("d_w_pre", "d_w_post", "d_gate"):
        got, want = host(big[n]), times * host(s[n])
        bound = 2.0 ** -7 * np.abs(want) + (T * times / 256 + 96) * U * T * times
        assert (np.abs(got - want) <= bound).all(), n
