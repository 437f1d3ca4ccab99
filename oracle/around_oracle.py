"""Oracle of the operators around the layer (NumPy, float64): the router's auxiliary losses and their gradients, the
norms with gate and residual scales, and the orthogonalised update.  Written from the formulas, independently of the
GPU path.

Sources: PLENA_Compiler PR #69, sections "Group B" (residual_setup) and "Group E" (the router's logits and top-k);
VeOmni docs "Fused MoE Kernel Notes", section "Duplicate top-k routes" (each slot counts)."""

from __future__ import annotations

import numpy as np

from oracle.train_oracle import route_backward

F = np.float64


def log_sum_exp(logits):
    top = logits.max(axis=1, keepdims=True)
    return (top + np.log(np.exp(logits - top).sum(axis=1, keepdims=True)))[:, 0]


def balance_loss(logits, ids, mask, top_k, balance_coef, z_coef):
    """(losses [2], counts [E], tokens, prob_sums [E], lse [T]); mask None: every token is valid."""
    logits = np.asarray(logits, F)
    T, E = logits.shape
    valid = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    lse, counts, sums = np.zeros(T), np.zeros(E, np.int64), np.zeros(E)
    if valid.any():
        lse[valid] = log_sum_exp(logits[valid])
        sums = np.exp(logits[valid] - lse[valid, None]).sum(axis=0)
    for t in np.flatnonzero(valid):
        for e in ids[t]:
            if 0 <= e < E:
                counts[e] += 1
    n = max(int(valid.sum()), 1)
    balance = balance_coef * E / (top_k * n * n) * float((counts * sums).sum())
    z = z_coef / n * float((lse[valid] ** 2).sum())
    return np.array([balance, z]), counts, int(valid.sum()), sums, lse


def balance_d_logits(logits, lse, mask, counts, tokens, top_k, balance_coef, z_coef):
    """Gradient [T, E] of the two losses' sum in the logits, counts held fixed."""
    logits, lse, c = np.asarray(logits, F), np.asarray(lse, F), np.asarray(counts, F)
    T, E = logits.shape
    n = max(int(tokens), 1)
    valid = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    d = np.zeros((T, E))
    rows = logits[valid]
    p = np.exp(rows - log_sum_exp(rows)[:, None]) if len(rows) else rows   # lse may be rounded to float32
    d[valid] = p * (balance_coef * E / (top_k * n * n) * (c - (p * c).sum(axis=1, keepdims=True))
                    + 2 * z_coef / n * lse[valid, None])
    return d


def route_balance_backward(x, w_router, logits, lse, ids, weights, d_weights, mask, counts, tokens, top_k,
                           balance_coef, z_coef):
    """(d_x, d_w_router, d_logit_bias, d_logits); weights and d_weights may both be None."""
    x, wr = np.asarray(x, F), np.asarray(w_router, F)
    d = balance_d_logits(logits, lse, mask, counts, tokens, top_k, balance_coef, z_coef)
    if weights is not None:
        d = d + route_backward(x, wr, ids, weights, d_weights)[3]
    return d @ wr.T, x.T @ d, d.sum(axis=0), d


def rstd(v, eps):
    return 1.0 / np.sqrt((np.asarray(v, F) ** 2).mean(axis=1) + eps)


def norm_residual(h, y=None, w_post=None, gate=None, eps=1e-6, offset=0.0, rs=1.0, bs=1.0):
    """(h_out, rstd_post): the stream after the branch, not rounded (y None: h itself)."""
    h = np.asarray(h, F)
    if y is None:
        return h, None
    n, r = np.asarray(y, F), None
    if w_post is not None:
        r = rstd(n, eps)
        n = n * r[:, None] * (offset + np.asarray(w_post, F))
    if gate is not None:
        n = n * np.asarray(gate, F)
    return rs * h + bs * n, r


def norm(h_out, w_pre, eps=1e-6, offset=0.0):
    """(x, rstd_pre) of the stream as stored."""
    r = rstd(h_out, eps)
    return np.asarray(h_out, F) * r[:, None] * (offset + np.asarray(w_pre, F)), r


def norm_backward(d, v, r, w, offset):
    """(gradient of v * r * (offset + w) in v, in w), r depending on v."""
    v, r, w, d = (np.asarray(a, F) for a in (v, r, w, d))
    hat, g = v * r[:, None], d * (offset + w)
    return r[:, None] * (g - hat * (g * hat).mean(axis=1, keepdims=True)), (d * hat).sum(axis=0)


def norm_residual_backward(d_h_out, d_x, h_out, rstd_pre, w_pre, y, rstd_post, w_post, gate, branch, offset=0.0,
                           rs=1.0, bs=1.0):
    """{d_h, d_y, d_w_pre, d_w_post, d_gate}; d_h_out, d_x and the weights may be None."""
    out = dict.fromkeys(("d_h", "d_y", "d_w_pre", "d_w_post", "d_gate"))
    d = 0.0 if d_h_out is None else np.asarray(d_h_out, F)
    if d_x is not None:
        g, out["d_w_pre"] = norm_backward(d_x, h_out, rstd_pre, w_pre, offset)
        d = d + g
    if not branch:
        out["d_h"] = d
        return out
    out["d_h"] = rs * d
    d_n = bs * d
    if gate is not None:
        n = np.asarray(y, F)
        if w_post is not None:
            n = n * np.asarray(rstd_post, F)[:, None] * (offset + np.asarray(w_post, F))
        out["d_gate"] = (d_n * n).sum(axis=0)
        d_n = d_n * np.asarray(gate, F)
    if w_post is not None:
        out["d_y"], out["d_w_post"] = norm_backward(d_n, y, rstd_post, w_post, offset)
    else:
        out["d_y"] = d_n
    return out


def orthogonalise(g, coefs, eps=1e-7):
    """The matrix after the Newton-Schulz steps."""
    x = np.asarray(g, F)
    x = x / (np.sqrt((x ** 2).sum()) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for a, b, c in coefs:
        gram = x @ x.T
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.T if tall else x


def orthogonal_update(grad, out, momentum=None, mu=0.95, nesterov=True, parts=1, coefs=(), eps=1e-7, scale=1.0,
                      keep=0.0):
    """(out, momentum) after a step; grad, out and momentum are [batch, M, parts * N]."""
    grad = np.asarray(grad, F)
    u, m = grad, None
    if momentum is not None:
        m = mu * np.asarray(momentum, F) + grad
        u = grad + mu * m if nesterov else m
    N = grad.shape[2] // parts
    res = np.empty_like(grad)
    for i in range(grad.shape[0]):
        for j in range(parts):
            cols = slice(j * N, (j + 1) * N)
            res[i, :, cols] = scale * orthogonalise(u[i, :, cols], coefs, eps)
    return (res if keep == 0.0 else keep * np.asarray(out, F) + res), m
