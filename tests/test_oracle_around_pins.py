"""Pins of the oracle of the operators around the layer: closed forms, invariants and gradients against differences."""

import numpy as np
import pytest

from oracle import around_oracle as O

COEFS = ((3.4445, -4.7750, 2.0315),) * 5


def rng(seed):
    return np.random.default_rng(seed)


def difference(f, v, d, h=1e-6):
    """Directional derivative of f at v along d."""
    return (f(v + h * d) - f(v - h * d)) / (2 * h)


def test_even_routes_have_balance_loss_one():
    T, E, k = 12, 4, 2
    ids = np.array([[t % E, (t + 1) % E] for t in range(T)])
    losses, counts, n, sums, lse = O.balance_loss(np.zeros((T, E)), ids, None, k, 1.0, 1.0)
    assert counts.tolist() == [6] * 4 and n == T
    assert np.allclose(losses, [1.0, np.log(E) ** 2]) and np.allclose(sums, T / E) and np.allclose(lse, np.log(E))


def test_one_expert_takes_all():
    T, E, k = 5, 8, 2
    logits = np.full((T, E), -1e9)
    logits[:, 3] = 0.0
    losses, counts, *_ = O.balance_loss(logits, np.full((T, k), 3), None, k, 1.0, 0.0)
    assert counts[3] == T * k and counts.sum() == T * k and np.isclose(losses[0], E)


def test_masked_tokens_and_wrong_ids_count_nowhere():
    r = rng(0)
    logits, ids = r.normal(size=(6, 4)), r.integers(0, 4, (6, 2))
    ids[1, 0] = 9
    mask = np.array([1, 1, 0, 1, 0, 1])
    a = O.balance_loss(logits, ids, mask, 2, 0.5, 0.25)
    keep = mask.astype(bool)
    b = O.balance_loss(logits[keep], ids[keep], None, 2, 0.5, 0.25)
    assert np.allclose(a[0], b[0]) and (a[1] == b[1]).all() and a[2] == 4 and a[1].sum() == 7
    assert (a[4][~keep] == 0).all()
    nothing = O.balance_loss(logits, ids, np.zeros(6), 2, 0.5, 0.25)
    assert (nothing[0] == 0).all() and nothing[2] == 0 and (nothing[1] == 0).all() and (nothing[3] == 0).all()


@pytest.mark.parametrize("masked", [False, True])
def test_balance_gradient_against_differences(masked):
    r = rng(1)
    T, E, k = 7, 5, 2
    logits, ids = r.normal(size=(T, E)), r.integers(0, E, (T, k))
    mask = np.array([1, 0, 1, 1, 0, 1, 1]) if masked else None
    _, counts, n, _, lse = O.balance_loss(logits, ids, mask, k, 0.3, 0.2)
    d = O.balance_d_logits(logits, lse, mask, counts, n, k, 0.3, 0.2)
    for _ in range(4):
        v = r.normal(size=logits.shape)
        want = difference(lambda z: O.balance_loss(z, ids, mask, k, 0.3, 0.2)[0].sum(), logits, v)
        assert np.isclose((d * v).sum(), want, rtol=1e-6)


def test_route_gradients_against_differences():
    r = rng(2)
    T, H, E, k = 6, 8, 5, 2
    x, w, bias = r.normal(size=(T, H)), r.normal(size=(H, E)), r.normal(size=E)
    ids = np.argsort(-(x @ w + bias), axis=1)[:, :k]
    dw = r.normal(size=(T, k))
    mask = np.array([1, 1, 0, 1, 1, 1])

    def parts(x, w, bias):
        logits = x @ w + bias
        sel = np.take_along_axis(logits, ids, 1)
        q = np.exp(sel - sel.max(1, keepdims=True))
        return logits, q / q.sum(1, keepdims=True)

    def loss(x, w, bias):
        logits, q = parts(x, w, bias)
        return (q * dw).sum() + O.balance_loss(logits, ids, mask, k, 0.7, 0.1)[0].sum()

    logits, q = parts(x, w, bias)
    _, counts, n, _, lse = O.balance_loss(logits, ids, mask, k, 0.7, 0.1)
    d_x, d_w, d_b, _ = O.route_balance_backward(x, w, logits, lse, ids, q, dw, mask, counts, n, k, 0.7, 0.1)
    for g, i in ((d_x, 0), (d_w, 1), (d_b, 2)):
        v = r.normal(size=g.shape)

        def along(s):
            a = [x, w, bias]
            a[i] = s
            return loss(*a)

        assert np.isclose((g * v).sum(), difference(along, [x, w, bias][i], v), rtol=1e-6)


@pytest.mark.parametrize("post,gated,pre", [(1, 1, 1), (0, 1, 1), (1, 0, 1), (0, 0, 1), (1, 1, 0)])
def test_norm_gradients_against_differences(post, gated, pre):
    r = rng(3)
    T, H = 4, 16
    a = {"h": r.normal(size=(T, H)), "y": r.normal(size=(T, H)), "w_post": r.normal(size=H) if post else None,
         "gate": r.normal(size=H) if gated else None, "w_pre": r.normal(size=H) if pre else None}
    kw = dict(eps=1e-5, offset=0.5, rs=0.9, bs=0.3)
    d_out, d_x = r.normal(size=(T, H)), r.normal(size=(T, H)) if pre else None

    def loss(a):
        h_out, _ = O.norm_residual(a["h"], a["y"], a["w_post"], a["gate"], **kw)
        v = (h_out * d_out).sum()
        return v + (O.norm(h_out, a["w_pre"], 1e-5, 0.5)[0] * d_x).sum() if pre else v

    h_out, r_post = O.norm_residual(a["h"], a["y"], a["w_post"], a["gate"], **kw)
    r_pre = O.norm(h_out, a["w_pre"], 1e-5, 0.5)[1] if pre else None
    g = O.norm_residual_backward(d_out, d_x, h_out, r_pre, a["w_pre"], a["y"], r_post, a["w_post"], a["gate"], True,
                                 0.5, 0.9, 0.3)
    for name, grad in (("h", "d_h"), ("y", "d_y"), ("w_post", "d_w_post"), ("gate", "d_gate"), ("w_pre", "d_w_pre")):
        if a[name] is None:
            assert g[grad] is None
            continue
        v = r.normal(size=a[name].shape)
        want = difference(lambda s, n=name: loss({**a, n: s}), a[name], v)
        assert np.isclose((g[grad] * v).sum(), want, rtol=1e-5), name


def test_norm_without_branch():
    r = rng(4)
    h, w = r.normal(size=(3, 8)), r.normal(size=8)
    x, q = O.norm(h, w)
    assert np.allclose((x / w) ** 2 @ np.ones(8) / 8, 1.0, atol=1e-5)
    d_x, d_out = r.normal(size=(3, 8)), r.normal(size=(3, 8))
    g = O.norm_residual_backward(d_out, d_x, h, q, w, None, None, None, None, False, rs=5.0)
    alone = O.norm_residual_backward(None, d_x, h, q, w, None, None, None, None, False)
    assert np.allclose(g["d_h"], d_out + alone["d_h"]) and g["d_y"] is None


@pytest.mark.parametrize("M,N", [(6, 10), (10, 6), (8, 8), (1, 5), (5, 1), (1, 1)])
def test_orthogonalised_keeps_singular_vectors(M, N):
    g = rng(5).normal(size=(M, N))
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((s ** 2).sum()) + 1e-7)
    for a, b, c in COEFS:
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(O.orthogonalise(g, COEFS), u @ np.diag(s) @ vt, atol=1e-10)
    assert (s > 0.6).all() and (s < 1.2).all()


def test_orthogonal_update_parts_momentum_and_keep():
    r = rng(6)
    g, w, m = (r.normal(size=(2, 4, 6)) for _ in range(3))
    out, mom = O.orthogonal_update(g, w, m, 0.9, True, 2, COEFS, 1e-7, -0.1, 0.5)
    m1 = 0.9 * m + g
    want = 0.5 * w[1, :, 3:] - 0.1 * O.orthogonalise((g + 0.9 * m1)[1, :, 3:], COEFS)
    assert np.allclose(out[1, :, 3:], want) and np.allclose(mom, m1)
    plain, none = O.orthogonal_update(g, w, coefs=COEFS)
    assert none is None and np.allclose(plain[0], O.orthogonalise(g[0], COEFS))
    assert (O.orthogonalise(np.zeros((3, 4)), COEFS) == 0).all()
