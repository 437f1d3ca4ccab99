"""GPU tests of the training calls at the edges of their ranges: values next to the types' limits, token counts next to
the launch limits, lists longer than a launch's table.  Bounds as in test_gpu_train: sums of K fp32 products within
4 (K + 16) 2^-24 of the magnitudes, half a step for a store."""

import numpy as np
import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B
from mixture_experts_ffn_05_amd import workloads as wl
from oracle import moe_oracle as O
from oracle import train_oracle as TO
from tests.gpu_helpers import host
from tests.test_gpu_train import DEV, GUARD, LAYERS, TORCH, U, Out, check, dev, grad_list, layer_step
from tests.test_gpu_train import test_route_backward as check_route_backward
from tests.test_gpu_train import test_shared_backward as check_shared_backward
from tests.test_gpu_train import test_shared_forward as check_shared_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.load()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu_gradient_where_partial_products_leave_fp32(dtype):
    """d_h is finite wherever its value is, also where da * u or da * g overflows: u = 1e30 and da = 1e20 or 3e37 with
    gates so negative that the sigmoid brings the product back, down to one that rounds to 0."""
    td = TORCH[dtype]
    rnd = O.bf16_rne if dtype == "bf16" else (lambda a: np.asarray(a, np.float32))
    T, H, I_s = 3, 8, 8
    g = rnd(np.array([-200, -104, -90, -80, -60, -46, -40, -33], np.float32))
    u = rnd(np.full(I_s, 1e30, np.float32))
    h = np.tile(np.concatenate([g, u]), (T, 1)).astype(np.float32)
    h[2, I_s:] = 1.0
    dy = np.zeros((T, H), np.float32)
    dy[:, 3] = rnd(np.array([1e20, -1e20, 3e37], np.float32))
    ws2 = torch.zeros((I_s, H), dtype=td, device=DEV)
    ws2[:, 3] = 1.0
    d_h, d_ws2 = Out((T, 2 * I_s), td), Out((I_s, H), td)
    ws = torch.zeros((B.moe_shared_train_workspace_bytes(td, T, H, I_s),), dtype=torch.uint8, device=DEV)
    B.moe_shared_fc2_backward(dev(dy), torch.zeros((T, I_s), dtype=td, device=DEV), dev(h, td), ws2, None, None, d_h.t,
                              d_ws2.t, None, ws)
    torch.cuda.synchronize()
    z, up, da = h[:, :I_s].astype(np.float64), h[:, I_s:].astype(np.float64), dy[:, 3:4].astype(np.float64)
    s = 1 / (1 + np.exp(-z))
    want = np.concatenate([da * up * s * (1 + z * (1 - s)), da * z * s], axis=1)
    assert np.abs(want).max() < 3e38
    mag = np.concatenate([np.abs(da * up) * s * (1 + np.abs(z)), np.abs(da * z) * s], axis=1)
    # a sigmoid below the normal numbers (2^-126) may count as 0
    far = 2.0 ** -126 * np.concatenate([np.abs(da * up) * (1 + np.abs(z)), np.abs(da * z)], axis=1) * \
        (np.tile(s, 2) < 2.0 ** -125)
    # the exponent's argument is an fp32 number of size 1.45 |z|: |z| 2^-24 relative on top of the few roundings
    check(d_h.get(), want, (16 + 2 * np.tile(np.abs(z), 2)) * U * mag + far, dtype, "d_h")


def fro(a, b):
    return float((a - b).norm() / b.norm())


# half a step of bf16 is 2^-8 of a value or less, evenly spread: 2^-8 / sqrt(3) on average (root mean square), and two
# independent roundings add in squares
TWO_ROUNDINGS = 2.0 ** -8 * (2.0 / 3.0) ** 0.5


@pytest.mark.parametrize("layout", [B.MOE_W_KN, B.MOE_W_NK], ids=["kn", "nk"])
@pytest.mark.parametrize("T,H,I,gated", [(517, 2048, 2816, False), (1021, 1024, 1408, True)])
def test_fc2_backward_is_two_roundings_from_the_formula(T, H, I, gated, layout):
    """Against float64 without any rounding: gate * dy is rounded for the products and the results are stored, each once;
    and the call gives the same bits again, whatever its workspace and outputs held."""
    D, bf = torch.float64, torch.bfloat16
    gen = torch.Generator(device=DEV).manual_seed(T + H)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)   # noqa: E731
    put = lambda w: w if layout == B.MOE_W_KN else w.t().contiguous()   # noqa: E731
    kn = lambda w: w if layout == B.MOE_W_KN else w.t()                 # noqa: E731
    dy, act, h, ws2 = rnd(T, H), rnd(T, I).to(bf), rnd(T, 2 * I).to(bf), (rnd(I, H) * I ** -0.5).to(bf)
    ys, gate = (rnd(T, H), torch.sigmoid(rnd(T))) if gated else (None, None)
    ws = torch.empty((B.moe_shared_train_workspace_bytes(bf, T, H, I),), dtype=torch.uint8, device=DEV)
    runs = []
    for r in range(3):
        d_h, d_w = torch.full((T, 2 * I), float(r), dtype=bf, device=DEV), torch.full_like(put(ws2), float(r))
        d_z = torch.full((T,), float(r), device=DEV) if gated else None
        ws.random_(0, 256)
        B.moe_shared_fc2_backward(dy, act, h, put(ws2), ys, gate, d_h, d_w, d_z, ws, layout=layout)
        torch.cuda.synchronize()
        runs.append([t for t in (d_h, d_w, d_z) if t is not None])
    for again in runs[1:]:
        for a, b in zip(again, runs[0]):
            assert torch.equal(a, b)
    rows = dy.to(D) * gate.to(D)[:, None] if gated else dy.to(D)
    da, mag = torch.mm(rows, ws2.to(D).t().contiguous()), torch.mm(rows.abs(), ws2.to(D).abs().t().contiguous())
    g, u = h[:, :I].to(D), h[:, I:].to(D)
    s = torch.sigmoid(g)
    half = 2.0 ** -8
    for got, want, factor in ((d_h[:, :I], da * u * s * (1 + g * (1 - s)), u.abs() * s * (1 + g.abs() * (1 - s))),
                              (d_h[:, I:], da * g * s, g.abs() * s)):
        err = (got.to(D) - want).abs()
        tol = factor * mag * (half + 4 * (H + 32) * U) * (1 + half) + half * want.abs() + 1e-37
        assert int((~(err <= tol)).sum()) == 0, float((err / tol).max())
        assert fro(got.to(D), want) <= TWO_ROUNDINGS
    want = torch.mm(act.to(D).t().contiguous(), rows)
    mag = torch.mm(act.to(D).abs().t().contiguous(), rows.abs())
    err = (kn(d_w).to(D) - want).abs()
    assert int((~(err <= mag * (half + 4 * (T + 16) * U) * (1 + half) + half * want.abs())).sum()) == 0
    assert fro(kn(d_w).to(D), want) <= TWO_ROUNDINGS


@pytest.mark.parametrize("T,H,E,k", [(1021, 2048, 60, 4), (1000, 1024, 256, 8)])
def test_route_backward_is_two_roundings_from_the_formula(T, H, E, k):
    """As above for d_w_router (d_logits is rounded for its product); d_x and the bias take the unrounded d_logits."""
    D, bf = torch.float64, torch.bfloat16
    gen = torch.Generator(device=DEV).manual_seed(T + E)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)   # noqa: E731
    x, wr = rnd(T, H).to(bf), (0.02 * rnd(H, E)).to(bf)
    top, ids = rnd(T, E).topk(k, dim=1)
    w, dw, dx0 = torch.softmax(top, dim=1).contiguous(), rnd(T, k), rnd(T, H)
    ids = ids.to(torch.int32).contiguous()
    ws = torch.empty((B.moe_route_backward_workspace_bytes(bf, T, H, E, k),), dtype=torch.uint8, device=DEV)
    runs = []
    for r in range(3):
        d_x, d_wr = dx0.clone(), torch.full((H, E), float(r), dtype=bf, device=DEV)
        d_b = torch.full((E,), float(r), device=DEV)
        ws.random_(0, 256)
        B.moe_route_backward(x, wr, ids, w, dw, d_x, d_wr, d_b, ws, accumulate=True)
        torch.cuda.synchronize()
        runs.append([d_x, d_wr, d_b])
    for again in runs[1:]:
        for a, b in zip(again, runs[0]):
            assert torch.equal(a, b)
    p, dp = w.to(D), dw.to(D)
    dl = p * (dp - (p * dp).sum(1, keepdim=True))
    dlm = p * (dp.abs() + (p * dp.abs()).sum(1, keepdim=True)) * 4 * (2 * k + 16) * U     # its fp32 evaluation
    dense, slack = (torch.zeros((T, E), dtype=D, device=DEV).scatter_(1, ids.long(), v) for v in (dl, dlm))
    half = 2.0 ** -8
    want, xa = torch.mm(x.to(D).t().contiguous(), dense), x.to(D).abs().t().contiguous()
    err = (d_wr.to(D) - want).abs()
    tol = torch.mm(xa, dense.abs() * (half + 4 * (T + 16) * U) * (1 + half) + slack) * (1 + half) + half * want.abs()
    assert int((~(err <= tol)).sum()) == 0, float((err / tol).max())
    assert fro(d_wr.to(D), want) <= TWO_ROUNDINGS
    wrt = wr.to(D).t().contiguous()
    want = dx0.to(D) + torch.mm(dense, wrt)
    tol = torch.mm(slack + dense.abs() * 4 * (k + 16) * U, wrt.abs()) + 4 * U * dx0.to(D).abs() + U * want.abs()
    assert int((~((d_x.to(D) - want).abs() <= tol)).sum()) == 0
    want = dense.sum(0)
    tol = (slack + dense.abs() * 4 * (T + 16) * U).sum(0)
    assert int((~((d_b.to(D) - want).abs() <= tol)).sum()) == 0


def test_more_tokens_than_a_launch_has_waves():
    """2^26 + 5 tokens, 8 wide: a wave per token would pass the 2^32 - 1 threads of a launch.  dy is zero but for some
    rows, so that every sum over the tokens has few terms."""
    T, H, I = (1 << 26) + 5, 8, 8
    D, bf = torch.float64, torch.bfloat16
    gen = torch.Generator(device=DEV).manual_seed(26)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)   # noqa: E731
    at = torch.cat([torch.tensor([0, 1, (1 << 24) - 1, 1 << 24, (1 << 26) - 1, 1 << 26, T - 1], device=DEV),
                    torch.randint(2, T - 1, (500,), generator=gen, device=DEV)]).unique()
    x, act, ws2, wg = rnd(T, H).to(bf), rnd(T, I).to(bf), rnd(I, H).to(bf), rnd(H).to(bf)
    ws = torch.empty((B.moe_shared_train_workspace_bytes(bf, T, H, I),), dtype=torch.uint8, device=DEV)
    nan = lambda *s, dt=torch.float32: torch.full(s, float("nan"), dtype=dt, device=DEV)   # noqa: E731
    y, ys, gate = nan(T, H), nan(T, H), nan(T)
    B.moe_shared_fc2_save(act, ws2, x, wg, y, ys, gate, ws)
    torch.cuda.synchronize()
    assert not gate.isnan().any() and not y.isnan().any() and not ys.isnan().any()
    a, xs = act[at].to(D), x[at].to(D)
    mag = torch.mm(a.abs(), ws2.to(D).abs())
    want, gt = torch.mm(a, ws2.to(D)), torch.sigmoid(torch.mv(xs, wg.to(D)))
    # one more rounding for each of the sums, the sigmoid's terms and the product with the gate
    zb = 4 * (H + 16) * U * torch.mv(xs.abs(), wg.to(D).abs()) / 4 + 8 * U * gt
    assert ((ys[at].to(D) - want).abs() <= 4 * (I + 16) * U * mag).all()
    assert ((gate[at].to(D) - gt).abs() <= zb).all()
    assert ((y[at].to(D) - gt[:, None] * want).abs() <= 4 * (I + 17) * U * mag + want.abs() * zb[:, None]).all()

    del x, y
    dy, h = torch.zeros((T, H), device=DEV), rnd(T, 2 * I).to(bf)
    dy[at] = rnd(at.numel(), H)
    d_h, d_w, d_z = nan(T, 2 * I, dt=bf), nan(I, H, dt=bf), nan(T)
    B.moe_shared_fc2_backward(dy, act, h, ws2, ys, gate, d_h, d_w, d_z, ws)
    torch.cuda.synchronize()
    g64, rows = gate[at].to(D), (gate[at][:, None] * dy[at]).to(bf).to(D)
    mag = (dy[at].to(D) * ys[at].to(D))
    tol = 4 * (H + 16) * U * mag.abs().sum(1) * g64 * (1 - g64)
    assert ((d_z[at].to(D) - g64 * (1 - g64) * mag.sum(1)).abs() <= tol).all()
    da, dab = torch.mm(rows, ws2.to(D).t().contiguous()), torch.mm(rows.abs(), ws2.to(D).abs().t().contiguous())
    g, u = h[at][:, :I].to(D), h[at][:, I:].to(D)
    s = torch.sigmoid(g)
    half = 2.0 ** -8
    for got, want, f in ((d_h[at][:, :I], da * u * s * (1 + g * (1 - s)), u.abs() * s * (1 + g.abs() * (1 - s))),
                         (d_h[at][:, I:], da * g * s, g.abs() * s)):
        assert ((got.to(D) - want).abs() <= 4 * (H + 24) * U * f * dab + half * want.abs() + 1e-37).all()
    am = act[at].to(D).t().contiguous()
    want = torch.mm(am, rows)
    assert ((d_w.to(D) - want).abs() <= 4 * (at.numel() + 16) * U * torch.mm(am.abs(), rows.abs())
            + half * want.abs()).all()
    d_h[at], d_z[at] = 0, 0
    assert not d_h.any() and not d_z.any()    # every other row: dy is zero, written as zeros


# A launch of the norm, or of scaling in place, takes 280 tensors, one of scaling into other tensors 180.
LONG = {"280": [5] * 280, "281": [5] * 280 + [9000], "181": [100] * 180 + [20000], "180": [8193] * 180,
        "600": [1 + 37 * i % 9001 for i in range(600)],
        # empty tensors on both sides of either table's end, and first and last
        "empty-edges": [0] + [30] * 177 + [0, 0, 0, 0] + [40] * 96 + [0, 0, 0, 0] + [8192] * 30 + [0],
        # tables of empty tensors only: the first (in place and out of place), one in the middle, the last
        "empty-first": [0] * 280 + [7, 8200], "empty-middle": [3] * 280 + [0] * 280 + [11, 12],
        "empty-last": [100000] + [0] * 600, "empty-all": [0] * 300}


@pytest.mark.parametrize("name", LONG)
def test_lists_longer_than_a_launch(name):
    """Norm, scaling into other tensors and scaling in place of lists that take several launches, against float64."""
    print(f"[case] {name}", flush=True)
    sizes = LONG[name]
    grads = grad_list(sizes, [0, 1, 3])
    h = [host(g).astype(np.float64) for g in grads]
    want = TO.grad_norm(h)
    lst = B.MoEGradList(grads)
    need = B.moe_grad_norm_workspace_bytes(lst.n)
    ws = torch.full((need + GUARD,), 255, dtype=torch.uint8, device=DEV)
    norm, sq = torch.full((1,), -1.0, device=DEV), torch.full((1,), -1.0, dtype=torch.float64, device=DEV)
    B.moe_grad_norm(lst, norm, ws[:need], sum_sq=sq)
    torch.cuda.synchronize()
    assert (ws[need:] == 255).all()
    assert abs(float(sq) - want ** 2) <= 1e-10 * want ** 2
    assert abs(float(norm) - want) <= 2 * U * want
    max_norm = 0.37 * want
    coef, c_in = torch.full((1,), -1.0, device=DEV), torch.full((1,), -1.0, device=DEV)
    outs = [Out((g.numel(),), g.dtype) for g in grads]
    B.moe_grad_clip(B.MoEGradList(grads, [o.t for o in outs]), norm, max_norm, coef)
    torch.cuda.synchronize()
    c = TO.clip_coef(float(norm), np.float32(max_norm).item())
    assert abs(float(coef) - c) <= 2 * U * c
    for g, v, o in zip(grads, h, outs):
        check(o.get(), v * float(coef), U * np.abs(v), "bf16" if g.dtype == torch.bfloat16 else "f32", name)
        np.testing.assert_array_equal(host(g).astype(np.float64), v)
    B.moe_grad_clip(lst, norm, max_norm, c_in)
    torch.cuda.synchronize()
    assert torch.equal(c_in, coef)
    for g, o in zip(grads, outs):
        assert torch.equal(g, o.t)
    # the factor of a list that needs none: 1, from the first launch only, and nothing moves
    B.moe_grad_clip(lst, norm, 1e30, c_in)
    torch.cuda.synchronize()
    assert float(c_in) == 1.0
    for g, o in zip(grads, outs):
        assert torch.equal(g, o.t)


def test_layer_gradients_match_differences_along_themselves():
    """Central differences of the float32 layer's forward along every parameter's own gradient, and of x along each term
    of its gradient (routed experts, router, shared expert, gate), where the derivative is as large as the gradient: a
    missing or doubled term shows.  A step of 1e-2 of a unit direction truncates by at most 1e-4 of the derivative (the
    oracle's forward in float64, every direction); y's fp32 sums are good to 1e-6 of each element, independently, and the
    step is what the stored parameters differ by."""
    cfg = LAYERS[2]
    layer = wl.make_layer(cfg, DEV)
    rng = np.random.default_rng(11)
    dy = rng.standard_normal((cfg.T, cfg.H)).astype(np.float32)
    bias = dev(np.array([30.0, 29.5, 0, -1, -2, -3])[: cfg.E])    # experts 0 and 1 for every token, a spread of weights
    bufs, tr = layer_step(cfg, B.MOE_W_KN, layer, dev(dy), bias)
    torch.cuda.synchronize()
    f64 = lambda t: host(t).astype(np.float64)   # noqa: E731
    w = f64(bufs.topk_weights)
    assert w.min() < 0.1 and set(host(bufs.topk_ids).ravel().tolist()) == {0, 1}
    ws1, ws2, wg = layer["shared"]
    params = {"d_x": layer["x"], "d_w_router": layer["w_router"], "d_w1": layer["W1"], "d_w2": layer["W2"],
              "d_ws1": ws1, "d_ws2": ws2, "d_w_gate": wg, "d_logit_bias": bias}
    grads = {n: f64(getattr(tr, n)).copy() for n in params}
    router = TO.route_backward(f64(layer["x"]), f64(layer["w_router"]), host(bufs.topk_ids), w, f64(tr.d_topk_weights))[0]
    gate, shared = np.outer(f64(tr.d_gate_logit), f64(wg)), f64(tr.d_h_shared) @ f64(ws1).T
    along = [(n, n, g) for n, g in grads.items()]
    along += [("d_x", "router", router), ("d_x", "gate", gate), ("d_x", "shared", shared),
              ("d_x", "routed", grads["d_x"] - router - gate - shared)]
    h = 1e-2
    noise = 1e-6 * np.sqrt(np.sum((dy * f64(bufs.y)) ** 2)) / h
    for name, what, d in along:
        p = params[name]
        keep, step, loss = p.clone(), [], []
        for sgn in (1, -1):
            p.copy_(keep + dev(sgn * h / np.linalg.norm(d) * d))
            step.append(f64(p).copy())
            b, _ = layer_step(cfg, B.MOE_W_KN, layer, dev(dy), bias)
            torch.cuda.synchronize()
            assert set(host(b.topk_ids).ravel().tolist()) == {0, 1}
            loss.append(np.sum(dy * f64(b.y)))
        p.copy_(keep)
        fd, an = (loss[0] - loss[1]) / (2 * h), np.sum(grads[name] * (step[0] - step[1])) / (2 * h)
        assert abs(fd - an) <= 2e-4 * abs(an) + 5 * noise, f"{what}: {fd} against {an} (rounding {noise})"
        # the term that the direction follows is far larger than what the comparison lets pass
        assert np.linalg.norm(d) > 100 * (2e-4 * abs(an) + 5 * noise), what


@pytest.mark.parametrize("layout", [B.MOE_W_KN, B.MOE_W_NK], ids=["kn", "nk"])
@pytest.mark.parametrize("size", [(1021, 1024, 704), (260, 2048, 1408), (2050, 264, 520), (3, 2048, 2816)],
                         ids=lambda s: "x".join(map(str, s)))
def test_float32_at_the_sizes_of_layers(size, layout):
    """The float32 calls past one tile, slice and chunk in every dimension, gated, both ways of accumulating."""
    check_shared_forward(size, "f32", True, layout)
    check_shared_backward(size, "f32", True, layout)


@pytest.mark.parametrize("case", [(1500, 1032, 200, 8, "f32"), (4100, 264, 64, 6, "f32")],
                         ids=lambda c: "x".join(map(str, c)))
def test_float32_router_at_the_sizes_of_layers(case):
    check_route_backward(case)


# from 65536 rows of 128 columns on a workgroup of d_x takes four tokens per thread; its pairs, 2 per thread up to 8
# slots a token, 8 beyond, and the weight product's tiles 64 or 128 experts wide
@pytest.mark.parametrize("case", [(8200, 1032, 64, 6, "bf16"), (8203, 1032, 60, 12, "bf16"), (8200, 1032, 100, 8, "bf16"),
                                  (8195, 1032, 100, 32, "bf16"), (8200, 1032, 64, 6, "f32"),
                                  (8203, 1032, 128, 12, "f32")], ids=lambda c: "x".join(map(str, c)))
def test_router_backward_of_many_tokens(case):
    check_route_backward(case)


@pytest.mark.parametrize("layout", [B.MOE_W_KN, B.MOE_W_NK], ids=["kn", "nk"])
@pytest.mark.parametrize("T,H,I", [(262149, 64, 4104), (262149, 8200, 64)], ids=["wide-h_pre", "wide-x"])
def test_tensors_past_two_to_the_31_elements(T, H, I, layout):
    """All four calls and the router's backward where a token tensor holds more than 2^31 elements: rows at both ends and
    at random against float64.  The incoming gradients are zero in every other row, so sums over tokens have few terms."""
    D, bf, f32 = torch.float64, torch.bfloat16, torch.float32
    gen = torch.Generator(device=DEV).manual_seed(T + H + layout)
    rnd = lambda *s, dt=bf, std=1.0: torch.randn(s, generator=gen, device=DEV, dtype=dt) * std   # noqa: E731
    new = lambda *s, dt=bf: torch.full(s, float("nan"), dtype=dt, device=DEV)                   # noqa: E731
    put = lambda w: w if layout == B.MOE_W_KN else w.t().contiguous()                           # noqa: E731
    kn = lambda w: w if layout == B.MOE_W_KN else w.t()                                         # noqa: E731
    at = torch.cat([torch.tensor([0, 1, T // 2, T - 2, T - 1], device=DEV),
                    torch.randint(2, T - 2, (200,), generator=gen, device=DEV)]).unique()
    n, half = at.numel(), 2.0 ** -8
    ws1, ws2, wg = rnd(H, 2 * I, std=H ** -0.5), rnd(I, H, std=I ** -0.5), rnd(H, std=H ** -0.5)
    ws = torch.empty((B.moe_shared_train_workspace_bytes(bf, T, H, I),), dtype=torch.uint8, device=DEV)
    mm = lambda a, b: torch.mm(a.to(D).contiguous(), b.to(D).contiguous())                      # noqa: E731
    bound = lambda a, b: 4 * (a.shape[1] + 16) * U * mm(a.abs(), b.abs())                       # noqa: E731

    def close(got, want, tol, store=half):
        err = (got.to(D) - want).abs()
        assert int((~(err <= tol + store * want.abs() + 1e-37)).sum()) == 0, float(err.max())

    x = rnd(T, H)
    act, h = new(T, I), new(T, 2 * I)
    B.moe_shared_fc1_save(x, put(ws1), act, h, ws, layout=layout)
    torch.cuda.synchronize()
    ref, hb = mm(x[at], ws1), bound(x[at], ws1)
    g, u = ref[:, :I], ref[:, I:]
    a = g * torch.sigmoid(g) * u
    close(h[at], ref, hb)
    close(act[at], a, 1.1 * hb[:, :I] * (u.abs() + hb[:, I:]) + g.abs() * hb[:, I:] + 16 * U * a.abs())
    y, ys, gate = new(T, H, dt=f32), new(T, H, dt=f32), new(T, dt=f32)
    B.moe_shared_fc2_save(act, put(ws2), x, wg, y, ys, gate, ws, layout=layout)
    torch.cuda.synchronize()
    ref, b = mm(act[at], ws2), bound(act[at], ws2)
    gt = torch.sigmoid(mm(x[at], wg[:, None]))[:, 0]
    gb = bound(x[at], wg[:, None])[:, 0] / 4 + 8 * U * gt
    close(ys[at], ref, b, U)
    close(gate[at], gt, gb, U)
    close(y[at], gt[:, None] * ref, b + ref.abs() * gb[:, None] + 4 * U * ref.abs(), U)
    assert not h.isnan().any() and not act.isnan().any() and not y.isnan().any() and not ys.isnan().any()
    del y
    dy = torch.zeros((T, H), device=DEV)
    dy[at] = rnd(n, H, dt=f32)
    d_h, d_w2, d_z = new(T, 2 * I), torch.full_like(put(ws2), float("nan")), new(T, dt=f32)
    B.moe_shared_fc2_backward(dy, act, h, put(ws2), ys, gate, d_h, d_w2, d_z, ws, layout=layout)
    torch.cuda.synchronize()
    rows, gd = (gate[at][:, None] * dy[at]).to(bf), gate[at].to(D)
    da, db = mm(rows, ws2.t()), bound(rows, ws2.t())
    g, u = h[at][:, :I].to(D), h[at][:, I:].to(D)
    s = torch.sigmoid(g)
    e = db + 16 * U * (da.abs() + db)
    close(d_h[at][:, :I], da * u * s * (1 + g * (1 - s)), u.abs() * s * (1 + g.abs() * (1 - s)) * e)
    close(d_h[at][:, I:], da * g * s, g.abs() * s * e)
    close(kn(d_w2), mm(act[at].t(), rows), bound(act[at].t(), rows))
    mag = dy[at].to(D) * ys[at].to(D)
    close(d_z[at], gd * (1 - gd) * mag.sum(1), 4 * (H + 16) * U * mag.abs().sum(1) * gd * (1 - gd), U)
    del dy, ys, h, act
    d_x, d_w1, d_wg = new(T, H, dt=f32), torch.full_like(put(ws1), float("nan")), new(H)
    B.moe_shared_fc1_backward(d_h, x, put(ws1), d_z, wg, d_x, d_w1, d_wg, ws, layout=layout)
    torch.cuda.synchronize()
    rank1 = d_z[at].to(D)[:, None] * wg.to(D)
    ref = mm(d_h[at], ws1.t())
    close(d_x[at], ref + rank1, bound(d_h[at], ws1.t()) + 8 * U * (ref.abs() + rank1.abs()), U)
    close(kn(d_w1), mm(x[at].t(), d_h[at]), bound(x[at].t(), d_h[at]))
    close(d_wg, mm(x[at].t(), d_z[at][:, None])[:, 0], bound(x[at].t(), d_z[at][:, None])[:, 0])
    for t in (d_h, d_x, d_z):
        t[at] = 0
        assert not t.any()          # every other row is written, as zeros
    del d_h, ws
    E, k = 16, 2
    wr, ids = rnd(H, E), torch.randint(0, E, (T, k), generator=gen, device=DEV, dtype=torch.int32)
    ids[:, 1] = (ids[:, 0] + 1 + ids[:, 1] % (E - 1)) % E      # two different experts
    w, dw = torch.full((T, k), 0.5, device=DEV), torch.zeros((T, k), device=DEV)
    dw[at] = rnd(n, k, dt=f32)
    rws = torch.empty((B.moe_route_backward_workspace_bytes(bf, T, H, E, k),), dtype=torch.uint8, device=DEV)
    d_wr, d_b = new(H, E), new(E, dt=f32)
    B.moe_route_backward(x, wr, ids, w, dw, d_x, d_wr, d_b, rws, accumulate=True)     # onto zeros
    torch.cuda.synchronize()
    q = dw[at].to(D)
    dl = 0.5 * (q - 0.5 * q.sum(1, keepdim=True))
    dlm = 4 * (2 * k + 16) * U * q.abs().sum(1, keepdim=True).expand(-1, k)
    dense, slack = (torch.zeros((n, E), dtype=D, device=DEV).scatter_(1, ids[at].long(), v) for v in (dl, dlm))
    close(d_x[at], mm(dense, wr.t()), mm(slack + 4 * (k + 16) * U * dense.abs(), wr.abs().t()), U)
    xa = x[at].to(D).abs().t()
    close(d_wr, mm(x[at].t(), dense), mm(xa, dense.abs() * (half + 4 * (n + 16) * U) + slack) * (1 + half))
    close(d_b, dense.sum(0), (slack + 4 * (n + 16) * U * dense.abs()).sum(0), U)
    d_x[at] = 0
    assert not d_x.any()


def test_scaling_partly_in_place_and_of_one_tensor_twice():
    """One list may scale some tensors in place and others into new ones, and may read one tensor for two outputs."""
    src = grad_list([9000, 20001, 77, 8192, 5], [0, 1, 3])
    keep = [g.clone() for g in src]
    norm = torch.full((1,), 4.0, device=DEV)
    outs = [src[0], torch.zeros_like(src[1]), src[2], torch.zeros_like(src[3]), torch.zeros_like(src[3]), src[4]]
    grads = [src[0], src[1], src[2], src[3], src[3], src[4]]
    for max_norm, factor in ((1.0, None), (100.0, 1.0)):
        before = [g.clone() for g in grads]
        coef = torch.zeros((1,), device=DEV)
        B.moe_grad_clip(B.MoEGradList(grads, outs), norm, max_norm, coef)
        torch.cuda.synchronize()
        c = float(coef)
        assert c == 1.0 if factor else abs(c - TO.clip_coef(4.0, 1.0)) <= 2 * U * c
        for b, o in zip(before, outs):
            v = host(b).astype(np.float64) * c
            check(host(o).astype(np.float64), v, U * np.abs(v), "bf16" if b.dtype == torch.bfloat16 else "f32", "out")
    assert torch.equal(src[1], keep[1]) and torch.equal(src[3], keep[3])
