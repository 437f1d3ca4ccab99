"""The operators around the layer against their formulas in float64.

Every bound counts roundings.  u is half a step of float32, 2^-24; a sum of n terms in any order is off by at most n u
times the sum of the terms' magnitudes; a stored bf16 value by half a step, 2^-8 of it."""

import numpy as np
import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B
from oracle import around_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def half(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def within(got, want, bound, what):
    """|got - want| <= bound, element by element; bound may be an array."""
    got, want = host(got), np.asarray(want)
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), f"{what}: off by {np.abs(got - want).max():.3e}, over the bound by {over.max():.3e}"


def ws(n):
    return torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------------------------------
# balance and z loss
# ------------------------------------------------------------------------------------------
def balance_state(T, E, k, mask, seed=0, spread=1.0):
    g = gen(seed)
    s = {"logits": normal(g, (T, E), spread) + normal(g, (E,), 0.7),
         "ids": torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)}
    s["mask"] = {None: None, "none": torch.zeros(T, dtype=torch.bool, device=DEV)}.get(mask) if mask in (None, "none") \
        else torch.rand((T,), generator=g, device=DEV) < 0.7
    s |= {"losses": torch.full((2,), 9.0, device=DEV), "prob_sums": torch.full((E,), 9.0, device=DEV),
          "counts": torch.full((E,), 9, dtype=torch.int32, device=DEV),
          "tokens": torch.full((1,), 9, dtype=torch.int32, device=DEV), "lse": torch.full((T,), 9.0, device=DEV)}
    s["ws"] = ws(B.moe_balance_loss_workspace_bytes(T, E))
    return s


def balance_call(s, coef=0.3, z=0.2, stream=None):
    B.moe_balance_loss(s["logits"], s["ids"], s["mask"], s["losses"], s["counts"], s["tokens"], s["prob_sums"], s["lse"],
                       s["ws"], coef, z, stream)


def check_balance(s, k, coef=0.3, z=0.2):
    mask = host(s["mask"])
    losses, counts, n, sums, lse = O.balance_loss(host(s["logits"]), s["ids"].cpu().numpy(), mask, k, coef, z)
    T, E = s["logits"].shape
    assert (s["counts"].cpu().numpy() == counts).all() and int(s["tokens"]) == n
    # exp and log within 2 ulp, an argument's rounding of its magnitude, a row's sum of E
    span = float(np.abs(host(s["logits"])).max()) * 2
    row = (E + 8 + span) * U
    within(s["lse"], lse, row + 4 * U * np.abs(lse), "lse")
    within(s["prob_sums"], sums, (row + (n + 8) * U) * sums, "prob_sums")
    top = np.abs(lse).max()
    within(s["losses"], losses, [(row + (n + E + 8) * U) * losses[0],
                                 (2 * row / max(top, 1e-3) + (n + 12) * U) * losses[1] + 2 * row * abs(z) * top],
           "losses")


@pytest.mark.parametrize("T,E,k,mask", [
    (1, 1, 1, None), (1, 4, 2, "some"), (3, 7, 7, None), (64, 8, 2, "some"), (65, 9, 3, None), (127, 16, 1, "some"),
    (130, 17, 4, None), (257, 33, 5, "some"), (1021, 60, 4, "some"), (300, 64, 6, None), (501, 65, 2, "some"),
    (77, 129, 8, None), (2000, 256, 8, "some"), (90, 255, 1, None), (33, 257, 8, "some"), (140, 512, 32, None),
    (19, 1000, 4, "some"), (21, 1024, 8, None), (20001, 8, 2, "some"), (9000, 130, 4, None), (16, 5, 2, "none")])
def test_balance_loss(T, E, k, mask):
    s = balance_state(T, E, k, mask, seed=T + E)
    balance_call(s)
    check_balance(s, k)


def test_balance_loss_duplicates_wrong_ids_and_far_logits():
    s = balance_state(100, 12, 3, "some", spread=40.0)
    s["ids"][::3] = 5                      # every slot names one expert
    s["ids"][1::3, 0] = -1
    s["ids"][2::3, 1] = 12
    s["logits"][4] = -3e38                 # the type's lowest values, all equal: an even softmax
    s["logits"][5, :6] = -float("inf")     # closed experts
    balance_call(s)
    mask = s["mask"].clone()
    bad = torch.zeros_like(mask)
    bad[4:6] = True
    assert torch.isfinite(s["losses"][:1]).all() and torch.isfinite(s["prob_sums"]).all()
    p = s["prob_sums"].double().sum().item()
    assert abs(p - int(s["tokens"])) <= 100 * 13 * U * 100
    keep = mask & ~bad
    s["mask"] = keep
    balance_call(s)
    check_balance(s, 3)


def test_masked_tokens_are_not_read():
    s = balance_state(70, 20, 2, "some")
    balance_call(s)
    want = {n: s[n].clone() for n in ("losses", "counts", "tokens", "prob_sums", "lse")}
    s["logits"][~s["mask"]] = float("nan")
    s["ids"][~s["mask"]] = 1 << 30
    balance_call(s)
    for n, v in want.items():
        assert torch.equal(s[n], v), n
    s["mask"] = s["mask"].to(torch.uint8) * 200   # any byte but 0
    balance_call(s)
    for n, v in want.items():
        assert torch.equal(s[n], v), n


# ------------------------------------------------------------------------------------------
# router backward with the losses
# ------------------------------------------------------------------------------------------
def route_state(T, H, E, k, dtype, mask, bias, seed=0):
    g = gen(seed)
    s = balance_state(T, E, k, mask, seed)
    balance_call(s)
    s["x"], s["wr"] = normal(g, (T, H), 1.0, dtype), normal(g, (H, E), 0.05, dtype)
    s["w"] = torch.softmax(normal(g, (T, k)), 1).contiguous()
    s["dw"] = normal(g, (T, k), 0.1)
    s["d_x"], s["old"] = normal(g, (T, H), 0.1), None
    s["old"] = s["d_x"].clone()
    s["d_wr"] = torch.full((H, E), 9.0, dtype=dtype, device=DEV)
    s["d_bias"] = torch.full((E,), 9.0, device=DEV) if bias else None
    s["rws"] = ws(B.moe_route_balance_backward_workspace_bytes(dtype, T, H, E, k))
    return s


def route_call(s, coef, z, accumulate, weights=True, stream=None):
    B.moe_route_balance_backward(s["x"], s["wr"], s["logits"], s["lse"], s["ids"], s["w"] if weights else None,
                                 s["dw"] if weights else None, s["mask"], s["counts"], s["tokens"], s["d_x"], s["d_wr"],
                                 s["d_bias"], s["rws"], coef, z, accumulate, stream)


def check_route(s, k, coef, z, accumulate, weights=True):
    T, H = s["x"].shape
    E = s["wr"].shape[1]
    dtype = s["x"].dtype
    mask, ids = host(s["mask"]), s["ids"].cpu().numpy()
    logits, lse, counts, n = host(s["logits"]), host(s["lse"]), host(s["counts"]), int(s["tokens"])
    w, dw = (host(s["w"]), host(s["dw"])) if weights else (None, None)
    x, wr = host(s["x"]), host(s["wr"])
    d_x, d_w, d_b, d = O.route_balance_backward(x, wr, logits, lse, ids, w, dw, mask, counts, n, k, coef, z)
    # what d's terms add up to in magnitude, and their roundings: exp's argument, the sums over experts and slots
    valid = np.ones(T, bool) if mask is None else mask.astype(bool)
    p = np.where(valid[:, None], np.exp(np.where(valid[:, None], logits - lse[:, None], 0.0)), 0.0)
    m = max(n, 1)
    mag = p * (abs(coef) * E / (k * m * m) * (counts + (p * counts).sum(1, keepdims=True))
               + 2 * abs(z) / m * np.abs(lse)[:, None])
    if weights:
        rows = np.arange(T)
        part = w * (np.abs(dw) + (w * np.abs(dw)).sum(1, keepdims=True))
        for j in range(k):
            np.add.at(mag, (rows, np.clip(ids[:, j], 0, E - 1)), part[:, j])
    d_err = (E + 2 * k + 24 + 4 * np.abs(logits).max()) * U * mag
    # the three (two) parts of a bf16 product leave 2^-24 (2^-16) of d; float32 products round each term
    left_x, left_w = (2.0 ** -24, 2.0 ** -16) if dtype == torch.bfloat16 else (0.0, 0.0)
    full = np.abs(d) + d_err
    old = host(s["old"]) if accumulate else 0.0
    within(s["d_x"], d_x + old,
           d_err @ np.abs(wr).T + (left_x + (3 * E + 16) * U) * (full @ np.abs(wr).T) + U * np.abs(old + d_x) * 2, "d_x")
    within(s["d_wr"], d_w, half(dtype) * np.abs(d_w)
           + (1 + half(dtype)) * (np.abs(x).T @ d_err + (left_w + (2 * T + 32) * U) * (np.abs(x).T @ full)), "d_w_router")
    if s["d_bias"] is not None:
        within(s["d_bias"], d_b, d_err.sum(0) + (T + 16) * U * full.sum(0), "d_logit_bias")


@pytest.mark.parametrize("T,H,E,k,dt,mask,bias,acc", [
    (1, 8, 1, 1, "bf16", None, True, False), (1, 64, 8, 2, "f32", None, False, True), (5, 72, 7, 3, "bf16", "some", True, True),
    (128, 256, 8, 2, "f32", "some", True, False), (130, 264, 60, 4, "bf16", "some", False, True),
    (257, 136, 64, 6, "bf16", None, True, False), (300, 512, 65, 2, "bf16", "some", True, True),
    (511, 128, 130, 8, "bf16", None, False, False), (1021, 256, 256, 8, "bf16", "some", True, True),
    (140, 64, 513, 4, "bf16", None, True, True), (70, 40, 1024, 32, "bf16", "some", True, False),
    (90, 48, 1000, 5, "f32", "some", True, True), (64, 1032, 16, 1, "bf16", "none", True, True),
    (4000, 128, 32, 4, "bf16", "some", True, True), (2000, 320, 96, 4, "f32", None, True, False)])
def test_route_balance_backward(T, H, E, k, dt, mask, bias, acc):
    s = route_state(T, H, E, k, TYPES[dt], mask, bias, seed=T + H)
    route_call(s, 0.7, 0.05, acc)
    check_route(s, k, 0.7, 0.05, acc)


@pytest.mark.parametrize("T,H,E,k,dt,mask", [
    (8192, 16, 12, 2, "bf16", "some"), (8193, 40, 60, 4, "bf16", "some"), (20001, 24, 130, 2, "bf16", None),
    (9000, 8, 300, 6, "f32", "some"), (8200, 16, 600, 3, "bf16", None)])
def test_route_balance_backward_of_many_tokens(T, H, E, k, dt, mask):
    s = route_state(T, H, E, k, TYPES[dt], mask, True, seed=T + E)
    route_call(s, 0.7, 0.05, True)
    check_route(s, k, 0.7, 0.05, True)


def test_losses_alone_and_wrong_ids():
    s = route_state(100, 64, 24, 3, torch.bfloat16, "some", True)
    route_call(s, 0.5, 0.1, False, weights=False)
    check_route(s, 3, 0.5, 0.1, False, weights=False)
    s["ids"][::2, 1] = 24
    s["ids"][1::2, 0] = -5
    s["ids"][3] = 7
    route_call(s, 0.5, 0.1, False)
    # the oracle drops those slots; magnitudes are counted at a neighbour, which only widens the bound
    check_route(s, 3, 0.5, 0.1, False)


def test_without_losses_as_the_plain_call():
    """Coefficients of zero: moe_route_backward's gradients (its d_w_router rounds d_logits once more)."""
    s = route_state(200, 128, 30, 4, torch.bfloat16, None, True)
    route_call(s, 0.0, 0.0, True)
    d_x, d_w, d_b = s["old"].clone(), torch.zeros_like(s["d_wr"]), torch.zeros_like(s["d_bias"])
    w = torch.empty((B.moe_route_backward_workspace_bytes(torch.bfloat16, 200, 128, 30, 4),), dtype=torch.uint8,
                    device=DEV)
    B.moe_route_backward(s["x"], s["wr"], s["ids"], s["w"], s["dw"], d_x, d_w, d_b, w, True)
    check_route(s, 4, 0.0, 0.0, True)
    assert torch.allclose(s["d_x"], d_x, rtol=0, atol=1e-5) and torch.allclose(s["d_bias"], d_b, rtol=0, atol=1e-5)
    assert torch.allclose(s["d_wr"].float(), d_w.float(), rtol=2 ** -6, atol=2e-2)


# ------------------------------------------------------------------------------------------
# norms and residual
# ------------------------------------------------------------------------------------------
EVERY = dict(branch=True, post=True, gate=True, pre=True)
KW = dict(weight_offset=0.5, residual_scale=0.9, branch_scale=0.3)


def norm_state(T, H, dtype, res, branch, post, gate, pre, seed=0):
    g = gen(seed)
    s = {"h": normal(g, (T, H), 1.5, res), "y": normal(g, (T, H), 0.7) if branch else None,
         "w_post": normal(g, (H,), 0.3, dtype) if post else None, "gate": normal(g, (H,), 0.6, dtype) if gate else None,
         "w_pre": normal(g, (H,), 0.3, dtype) if pre else None}
    nine = lambda shape, dt, want: torch.full(shape, 9.0, dtype=dt, device=DEV) if want else None   # noqa: E731
    f32 = torch.float32
    s |= {"h_out": nine((T, H), res, branch), "x": nine((T, H), dtype, pre), "rstd_post": nine((T,), f32, post),
          "rstd_pre": nine((T,), f32, pre), "d_h_out": normal(g, (T, H), 0.5, res),
          "d_x": normal(g, (T, H), 0.5) if pre else None, "d_h": nine((T, H), res, True),
          "d_y": nine((T, H), f32, branch), "d_w_pre": nine((H,), dtype, pre), "d_w_post": nine((H,), dtype, post),
          "d_gate": nine((H,), dtype, gate)}
    s["ws"] = ws(B.moe_norm_residual_backward_workspace_bytes(T, H))
    return s


def norm_forward(s, stream=None):
    B.moe_norm_residual(s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], s["h_out"], s["x"], s["rstd_post"],
                        s["rstd_pre"], 1e-6, stream=stream, **KW)


def norm_backward(s, stream=None):
    B.moe_norm_residual_backward(s["d_h_out"], s["d_x"], (s["h"] if s["h_out"] is None else s["h_out"]) if s["d_x"] is not None else None,
                                 s["rstd_pre"], s["w_pre"], s["y"], s["rstd_post"], s["w_post"], s["gate"], s["d_h"],
                                 s["d_y"], s["d_w_pre"], s["d_w_post"], s["d_gate"], s["ws"], stream=stream, **KW)


def check_norm_forward(s):
    H = s["h"].shape[1]
    off, rs, bs = KW.values()
    h, y, w_post, gate, w_pre = (host(s[n]) for n in ("h", "y", "w_post", "gate", "w_pre"))
    # a mean of H squares in any order, its root and reciprocal; the products after it
    r_err, chain = (H / 2 + 6) * U, (H / 2 + 16) * U
    if y is not None:
        h_out, r = O.norm_residual(h, y, w_post, gate, 1e-6, off, rs, bs)
        if r is not None:
            within(s["rstd_post"], r, r_err * r, "rstd_post")
        terms = np.abs(rs * h) + np.abs(h_out - rs * h) * (1.0 if w_post is None else 1.0) \
            + (0.0 if w_post is None else np.abs(bs * (1.0 if gate is None else gate) * y * r[:, None]) * (abs(off) + np.abs(w_post)))
        within(s["h_out"], h_out, half(s["h"].dtype) * np.abs(h_out) + (1 + half(s["h"].dtype)) * chain * terms, "h_out")
    if w_pre is not None:
        stored = host(s["h_out"]) if y is not None else h
        x, r = O.norm(stored, w_pre, 1e-6, off)
        within(s["rstd_pre"], r, r_err * r, "rstd_pre")
        mag = np.abs(stored) * r[:, None] * (abs(off) + np.abs(w_pre))
        within(s["x"], x, half(s["x"].dtype) * np.abs(x) + (1 + half(s["x"].dtype)) * chain * mag, "x")


def check_norm_backward(s):
    T, H = s["d_h"].shape
    off, rs, bs = KW.values()
    a = {n: host(s[n]) for n in ("d_h_out", "d_x", "h", "h_out", "rstd_pre", "w_pre", "y", "rstd_post", "w_post", "gate")}
    branch = s["d_y"] is not None
    stream = a["h"] if a["h_out"] is None else a["h_out"]
    want = O.norm_residual_backward(a["d_h_out"], a["d_x"], stream, a["rstd_pre"], a["w_pre"], a["y"], a["rstd_post"],
                                    a["w_post"], a["gate"], branch, off, rs, bs)
    # magnitudes: the same formulas of magnitudes, differences taken as sums; two means over H follow each other
    K = (2 * H + 64) * U
    d = 0.0 if a["d_h_out"] is None else np.abs(a["d_h_out"])
    sums = {}
    if a["d_x"] is not None:
        hat, g = np.abs(stream) * a["rstd_pre"][:, None], np.abs(a["d_x"]) * (abs(off) + np.abs(a["w_pre"]))
        d = d + a["rstd_pre"][:, None] * (g + hat * (g * hat).mean(1, keepdims=True))
        sums["d_w_pre"] = (np.abs(a["d_x"]) * hat).sum(0)
    t = s["d_h"].dtype
    within(s["d_h"], want["d_h"], half(t) * np.abs(want["d_h"]) + (1 + half(t)) * K * d * (rs if branch else 1.0), "d_h")
    if branch:
        gate = 1.0 if a["gate"] is None else np.abs(a["gate"])
        dn = bs * d * gate
        n = np.abs(a["y"])
        if a["w_post"] is not None:
            z, ow = n * a["rstd_post"][:, None], abs(off) + np.abs(a["w_post"])
            sums["d_w_post"] = (dn * z).sum(0)
            mag = a["rstd_post"][:, None] * (dn * ow + z * (dn * ow * z).mean(1, keepdims=True))
            n = z * ow
        else:
            mag = dn
        within(s["d_y"], want["d_y"], K * mag, "d_y")
        if a["gate"] is not None:
            sums["d_gate"] = (bs * d * n).sum(0)
    for name, mag in sums.items():
        w = s[name].dtype
        within(s[name], want[name], half(w) * np.abs(want[name]) + (1 + half(w)) * (K + (T + 32) * U) * mag, name)


PARTS = [EVERY, dict(branch=True, post=False, gate=True, pre=True), dict(branch=True, post=True, gate=False, pre=True),
         dict(branch=True, post=False, gate=False, pre=True), dict(branch=True, post=True, gate=True, pre=False),
         dict(branch=True, post=False, gate=False, pre=False), dict(branch=False, post=False, gate=False, pre=True)]


@pytest.mark.parametrize("parts", PARTS, ids=lambda p: "+".join(k for k, v in p.items() if v))
@pytest.mark.parametrize("dt,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_norm_parts_and_types(parts, dt, res):
    s = norm_state(37, 328, TYPES[dt], TYPES[res], **parts)
    norm_forward(s)
    check_norm_forward(s)
    norm_backward(s)
    check_norm_backward(s)


@pytest.mark.parametrize("T,H", [(1, 8), (1, 512), (2, 520), (3, 1024), (5, 1032), (1, 2048), (4, 2056), (7, 4096),
                                 (3, 4104), (9, 7168), (2, 8192), (1021, 64), (2100, 512), (1500, 1000), (700, 2048),
                                 (600, 4096), (300, 7168), (260, 8192)])
def test_norm_sizes(T, H):
    for dt, res in (("bf16", "bf16"), ("f32", "f32")):
        s = norm_state(T, H, TYPES[dt], TYPES[res], **EVERY, seed=T)
        norm_forward(s)
        check_norm_forward(s)
        norm_backward(s)
        check_norm_backward(s)


def test_norm_in_place_and_without_outer_gradient():
    s = norm_state(50, 264, torch.bfloat16, torch.bfloat16, **EVERY)
    norm_forward(s)
    norm_backward(s)
    h_out, x, d_h = s["h_out"].clone(), s["x"].clone(), s["d_h"].clone()
    h0, d0 = s["h"].clone(), s["d_h_out"].clone()
    s["h_out"] = s["h"]
    norm_forward(s)
    assert torch.equal(s["h"], h_out) and torch.equal(s["x"], x)
    s["d_h"] = s["d_h_out"]
    norm_backward(s)
    assert torch.equal(s["d_h_out"], d_h)
    s["h"], s["h_out"], s["d_h"] = h0, h_out, torch.empty_like(d0)
    s["d_h_out"] = None
    norm_backward(s)
    check_norm_backward(s)


def test_norm_rows_that_are_zero_or_not_finite():
    s = norm_state(8, 520, torch.bfloat16, torch.float32, **EVERY)
    s["h"][1] = 0
    s["y"][1] = 0                       # nothing: its norm is 0, not NaN
    s["y"][3, 5] = float("inf")
    s["h"][5, 7] = float("nan")
    norm_forward(s)
    assert (s["h_out"][1] == 0).all() and (s["x"][1] == 0).all()
    assert torch.isnan(s["x"][5]).all() and torch.isnan(s["x"][3]).any()
    fine = [0, 1, 2, 4, 6, 7]
    for n in ("h_out", "x"):
        assert torch.isfinite(s[n][fine].float()).all()


# ------------------------------------------------------------------------------------------
# orthogonalised update
# ------------------------------------------------------------------------------------------
QUINTIC = (3.4445, -4.7750, 2.0315)
COEFS = (QUINTIC,) * 5


def matrices(g, shape, kind, dtype):
    batch, M, N = shape
    if kind == "noise":
        v = normal(g, shape)
    else:   # a few strong directions over noise, as a batch's gradient
        v = torch.matmul(normal(g, (batch, M, 4)), normal(g, (batch, 4, N))) + normal(g, shape, 0.3)
    return (v * 1e-3).to(dtype)


def ortho_bound(dtype, n, steps=5):
    """Relative error of a result, 2-norms.  An operand's half step is 2^-12 of it in fp16 on average (2^-22 of it in
    two fp16, where a sum of n terms adds sqrt(n) 2^-24): three operands per step, independent, whose effect grows by
    at most the polynomial's slope a.  Then the result's own rounding, at most half a step."""
    each = 2.0 ** -12 if dtype == torch.bfloat16 else 2.0 ** -22 + n ** 0.5 * U
    return (3 * steps) ** 0.5 * QUINTIC[0] * each + half(dtype)


def ortho_call(grad, out, momentum=None, parts=1, stream=None, workspace=None, **kw):
    shape = grad.shape if grad.dim() == 3 else (1, *grad.shape)
    w = workspace if workspace is not None else ws(B.moe_orthogonal_update_workspace_bytes(
        grad.dtype, out.dtype, shape[0], shape[1], shape[2] // parts, parts, momentum is not None))
    B.moe_orthogonal_update(grad, out, w, momentum, parts=parts, stream=stream, **kw)
    return w


def rel(got, want):
    return float(np.linalg.norm(host(got) - want) / max(np.linalg.norm(want), 1e-300))


@pytest.mark.parametrize("M,N", [(1, 1), (1, 9), (8, 8), (7, 20), (20, 7), (32, 33), (33, 32), (60, 300), (300, 60),
                                 (64, 64), (65, 64), (100, 129), (128, 128), (128, 700), (900, 128), (129, 130),
                                 (131, 129), (136, 200), (200, 136), (129, 650), (700, 130), (256, 256), (264, 1400),
                                 (1400, 264), (300, 301), (400, 512)])
@pytest.mark.parametrize("kind", ["noise", "strong"])
def test_orthogonal_update_sizes(M, N, kind):
    g = gen(M * 7 + N)
    for dt in (torch.bfloat16, torch.float32):
        grad = matrices(g, (2, M, N), kind, dt)
        out = torch.full((2, M, N), 9.0, dtype=dt, device=DEV)
        ortho_call(grad, out)
        want, _ = O.orthogonal_update(host(grad), None, coefs=COEFS)
        bound = ortho_bound(dt, max(M, N))
        # noise that X's strong directions put on its small ones grows by a in every step but the last (float32 out)
        if dt == torch.float32 and kind == "strong":
            bound = bound * QUINTIC[0] ** 4
        assert rel(out, want) <= bound, dt


@pytest.mark.parametrize("dt,odt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("M,N,parts", [(24, 40, 2), (40, 24, 3), (130, 72, 2), (150, 160, 2), (700, 131, 1)])
def test_orthogonal_update_momentum_parts_keep(dt, odt, M, N, parts):
    g = gen(M + N)
    shape = (3, M, parts * N)
    grad, mom, w = matrices(g, shape, "strong", TYPES[dt]), normal(g, shape, 2e-3), normal(g, shape, 0.1, TYPES[odt])
    for nesterov in (True, False):
        want, want_m = O.orthogonal_update(host(grad), host(w), host(mom), 0.9, nesterov, parts, COEFS, 1e-7, -0.5, 0.75)
        ortho_call(grad, w, mom, parts, mu=0.9, nesterov=nesterov, scale=-0.5, keep=0.75)
        within(mom, want_m, 2 * U * (np.abs(want_m) + np.abs(host(grad))) + 1e-12, "momentum")
        bound = ortho_bound(w.dtype, max(M, N)) * (QUINTIC[0] ** 4 if odt == "f32" else 1)
        assert rel(w, want) <= bound


@pytest.mark.parametrize("M,N", [(40, 50), (200, 210), (140, 900)])
def test_other_coefficients(M, N):
    grad = matrices(gen(3), (1, M, N), "noise", torch.bfloat16)
    for coefs in (((1.5, -0.5, 0.0),), ((1.0, 0.0, 0.0),) * 3, ((4.0, -6.8, 3.0), (2.0, -1.5, 0.5)),
                  ((1.875, -1.25, 0.375),) * 16, ((0.0, 0.0, 0.0),)):
        out = torch.full_like(grad, 9.0)
        ortho_call(grad, out, coefs=coefs)
        want, _ = O.orthogonal_update(host(grad), None, coefs=coefs)
        if not want.any():
            assert (out == 0).all()
            continue
        slope = max(abs(a) for a, _, _ in coefs)
        assert rel(out, want) <= (3 * len(coefs)) ** 0.5 * max(slope, 1.0) * 2.0 ** -12 + 2.0 ** -8


@pytest.mark.parametrize("M,N", [(30, 50), (200, 150), (140, 900)])
def test_zero_tiny_large_and_broken_matrices(M, N):
    """Each matrix of a stack by itself: zeros stay zeros, one that is not finite is NaN throughout, scale is nothing."""
    g = gen(5)
    one = matrices(g, (1, M, N), "noise", torch.float32)
    grad = one.repeat(6, 1, 1)
    grad[0] = 0
    grad[1] *= 1e-9 / 1e-3
    grad[2] *= 2.0 ** 50
    grad[3, M // 2, N // 3] = float("nan")
    grad[4, 0, 0] = float("inf")
    for odt in (torch.bfloat16, torch.float32):
        out = torch.full(grad.shape, 9.0, dtype=odt, device=DEV)
        ortho_call(grad, out, eps=1e-12)
        assert (out[0] == 0).all() and torch.isnan(out[3]).all() and torch.isnan(out[4]).all()
        for i in (1, 2, 5):
            assert rel(out[i], O.orthogonalise(host(grad[i]), COEFS, 1e-12)) <= ortho_bound(odt, max(M, N)), i


def test_unaligned_tensors_and_what_lies_beside_them():
    """Views off any 16-byte boundary; a stack's neighbours keep their values."""
    g = gen(6)
    for M, N in ((30, 40), (150, 160)):
        store = normal(g, (2 * M * N + 16,), 1e-3, torch.bfloat16)
        res = torch.full((2 * M * N + 16,), 9.0, dtype=torch.bfloat16, device=DEV)
        grad, out = store[3:3 + 2 * M * N].view(2, M, N), res[5:5 + 2 * M * N].view(2, M, N)
        ortho_call(grad, out)
        want, _ = O.orthogonal_update(host(grad), None, coefs=COEFS)
        assert rel(out, want) <= ortho_bound(torch.bfloat16, N)
        assert (res[:5] == 9).all() and (res[5 + 2 * M * N:] == 9).all()


def test_two_dimensional_and_refusals():
    g = gen(7)
    grad = matrices(g, (1, 24, 36), "noise", torch.bfloat16)[0]
    out, same = torch.zeros_like(grad), torch.zeros((1, 24, 36), dtype=torch.bfloat16, device=DEV)
    w = ortho_call(grad, out)
    ortho_call(grad[None], same)
    assert torch.equal(out, same[0])
    with pytest.raises(B.MoEError, match="overlaps"):
        B.moe_orthogonal_update(grad, grad, w)
    with pytest.raises(ValueError, match="side by side"):
        B.moe_orthogonal_update(grad, out, w, parts=5)
    with pytest.raises(ValueError, match="three numbers"):
        B.moe_orthogonal_update(grad, out, w, coefs=[(1.0, 2.0)])
    with pytest.raises(B.MoEError, match="workspace needs"):
        B.moe_orthogonal_update(grad, out, w[:16])
    with pytest.raises(ValueError, match="shape"):
        B.moe_orthogonal_update(grad, out[:12], w)
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_orthogonal_update(grad.t(), out, w)
    with pytest.raises(TypeError, match="token_mask"):
        s = balance_state(4, 4, 1, None)
        s["mask"] = torch.ones(4, device=DEV)
        balance_call(s)


@pytest.mark.parametrize("M,N", [(30, 70), (40, 100), (100, 40), (120, 300), (200, 210), (140, 900), (900, 140)])
def test_many_steps_of_a_matrix_of_low_rank(M, N):
    """Few strong directions and none besides (whole numbers: exact in bf16), over more steps than five.  What the
    roundings of two fp16 planes put on the directions that are not there grows by a in every step but the last."""
    g = gen(M + N)
    ints = lambda shape: torch.randint(-3, 4, shape, generator=g, device=DEV).float()   # noqa: E731
    grad = torch.matmul(ints((2, M, 4)), ints((2, 4, N))).bfloat16()
    for steps in (6, 8, 12):
        out = torch.full_like(grad, 9.0)
        ortho_call(grad, out, coefs=(QUINTIC,) * steps)
        # the polynomial takes [0, 1.25] into [0, 1.21]
        for v in host(out):
            assert np.isfinite(v).all() and np.linalg.norm(v, 2) <= 1.25, steps
        if steps <= 8:
            want, _ = O.orthogonal_update(host(grad), None, coefs=(QUINTIC,) * steps)
            bound = ortho_bound(torch.float32, max(M, N), steps) * QUINTIC[0] ** (steps - 1) + half(torch.bfloat16)
            assert rel(out, want) <= bound, steps
