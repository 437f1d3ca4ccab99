"""Pins of the training oracle (CPU only): every gradient against central differences of the oracle's forward and
against PyTorch autograd in float64 through a formulation that shares no code with it."""

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from oracle import train_oracle as TO


def _shared_problem(gated, seed=5, T=7, H=16, I=24):
    rng = np.random.default_rng(seed)
    p = {"x": rng.standard_normal((T, H)), "ws1": rng.standard_normal((H, 2 * I)) / np.sqrt(H),
         "ws2": rng.standard_normal((I, H)) / np.sqrt(I)}
    if gated:
        p["w_gate"] = rng.standard_normal(H) / np.sqrt(H)
    return p, rng.standard_normal((T, H))


def _shared_y(p):
    act, _ = TO.shared_fc1(p["x"], p["ws1"])
    return TO.shared_fc2(act, p["ws2"], p["x"], p.get("w_gate"))[0]


def _shared_grads(p, dy):
    act, h = TO.shared_fc1(p["x"], p["ws1"])
    _, ys, gate = TO.shared_fc2(act, p["ws2"], p["x"], p.get("w_gate"))
    d_h, d_ws2, d_z = TO.shared_fc2_backward(dy, act, h, p["ws2"], ys, gate)
    d_x, d_ws1, d_wg = TO.shared_fc1_backward(d_h, p["x"], p["ws1"], d_z, p.get("w_gate"))
    return {"x": d_x, "ws1": d_ws1, "ws2": d_ws2, "w_gate": d_wg}


def test_shared_forward_is_the_layers_shared_expert():
    for gated in (False, True):
        p, _ = _shared_problem(gated)
        want = O.shared_expert(p["x"], p["ws1"], p["ws2"], p.get("w_gate"))
        np.testing.assert_allclose(_shared_y(p), want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("gated", [False, True])
def test_shared_gradients_match_central_differences(gated):
    p, dy = _shared_problem(gated)
    g = _shared_grads(p, dy)
    rng = np.random.default_rng(6)
    h = 1e-5
    for name in p:
        d = rng.standard_normal(p[name].shape)
        up, dn = ({**p, name: p[name] + s * h * d} for s in (1, -1))
        fd = np.sum(dy * (_shared_y(up) - _shared_y(dn))) / (2 * h)
        # truncation h^2 |f'''| and cancellation 2^-52 |f| / h, both under 1e-8 at these magnitudes
        np.testing.assert_allclose(np.sum(g[name] * d), fd, rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("gated", [False, True])
def test_shared_gradients_match_autograd(gated):
    p, dy = _shared_problem(gated, seed=8)
    t = {n: torch.tensor(v, requires_grad=True) for n, v in p.items()}
    half = p["ws2"].shape[0]
    y = torch.nn.functional.silu(t["x"] @ t["ws1"][:, :half]) * (t["x"] @ t["ws1"][:, half:]) @ t["ws2"]
    if gated:
        y = torch.sigmoid(t["x"] @ t["w_gate"])[:, None] * y
    y.backward(torch.tensor(dy))
    g = _shared_grads(p, dy)
    for n in p:
        np.testing.assert_allclose(g[n], t[n].grad.numpy(), rtol=1e-10, atol=1e-10)


def _route_problem(seed=9, T=9, H=8, E=6, k=3):
    rng = np.random.default_rng(seed)
    x, wr, b = rng.standard_normal((T, H)), rng.standard_normal((H, E)), rng.standard_normal(E)
    ids = np.argsort(-(x @ wr + b), axis=1)[:, :k].astype(np.int32)
    return x, wr, b, ids, rng.standard_normal((T, k))


def _selected_weights(x, wr, b, ids):
    logits = np.take_along_axis(x @ wr + b, np.clip(ids, 0, wr.shape[1] - 1), axis=1)
    e = np.exp(logits - logits.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def test_route_gradients_match_central_differences():
    x, wr, b, ids, dw = _route_problem()
    w = _selected_weights(x, wr, b, ids)
    d_x, d_wr, d_b, _ = TO.route_backward(x, wr, ids, w, dw)
    rng = np.random.default_rng(10)
    h = 1e-5
    f = lambda *a: np.sum(dw * _selected_weights(*a, ids))  # noqa: E731
    args = [x, wr, b]
    for i, grad in enumerate((d_x, d_wr, d_b)):
        d = rng.standard_normal(args[i].shape)
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * d, args[i] - h * d
        np.testing.assert_allclose(np.sum(grad * d), (f(*up) - f(*dn)) / (2 * h), rtol=1e-7, atol=1e-8)


def test_route_gradients_match_autograd_with_repeated_experts():
    x, wr, b, ids, dw = _route_problem(seed=12)
    ids[2, :] = ids[2, 0]              # every slot of one token names one expert
    ids[4, 1] = ids[4, 2]
    tx, twr, tb = (torch.tensor(v, requires_grad=True) for v in (x, wr, b))
    sel = torch.gather(tx @ twr + tb, 1, torch.tensor(ids.astype(np.int64)))
    w = torch.softmax(sel, dim=1)
    (w * torch.tensor(dw)).sum().backward()
    d_x, d_wr, d_b, d_logits = TO.route_backward(x, wr, ids, w.detach().numpy(), dw)
    np.testing.assert_allclose(d_x, tx.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(d_wr, twr.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(d_b, tb.grad.numpy(), rtol=1e-10, atol=1e-12)
    assert np.abs(d_logits[2]).max() < 1e-15   # one expert in every slot: its weights sum to 1 whatever the logit


def test_route_ids_outside_the_experts_reach_nothing():
    x, wr, b, ids, dw = _route_problem(seed=13)
    w = _selected_weights(x, wr, b, ids)
    ids2 = ids.copy()
    ids2[0, 1], ids2[3, 0] = -1, wr.shape[1]
    full = TO.route_backward(x, wr, ids, w, dw)[3]
    got = TO.route_backward(x, wr, ids2, w, dw)[3]
    want = full.copy()
    want[0, ids[0, 1]] = 0.0
    want[3, ids[3, 0]] = 0.0
    np.testing.assert_array_equal(got, want)


def test_norm_and_coefficient():
    assert TO.grad_norm([np.array([3.0]), np.array([[0.0, -4.0]])]) == 5.0
    assert TO.clip_coef(5.0, 10.0) == 1.0
    np.testing.assert_allclose(TO.clip_coef(5.0, 1.0), 0.2, rtol=1e-6)
    assert np.isnan(TO.clip_coef(np.nan, 1.0)) and TO.clip_coef(np.inf, 1.0) == 0.0
    assert TO.clip_coef(0.0, 0.0) == 0.0
    t = [torch.tensor([3.0, 1.0], dtype=torch.float64), torch.tensor([[0.5], [-4.0]], dtype=torch.float64)]
    params = [torch.nn.Parameter(torch.zeros_like(v)) for v in t]
    for p, v in zip(params, t):
        p.grad = v.clone()
    n = torch.nn.utils.clip_grad_norm_(params, 2.0)
    np.testing.assert_allclose(float(n), TO.grad_norm([v.numpy() for v in t]), rtol=1e-14)
    np.testing.assert_allclose(params[1].grad.numpy(), t[1].numpy() * TO.clip_coef(float(n), 2.0), rtol=1e-14)
