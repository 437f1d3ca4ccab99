"""Oracle of the layer's remaining training operators (NumPy, float64 unless asked otherwise): the shared expert's
training forward and backward, the router's backward, and the norm and clipping of a list of gradients.  Written from
the formulas, independently of the GPU path.

Sources: PLENA_Compiler PR #69, section "Group C -- shared experts" (the gated feed-forward block); PLENA_Simulator
PR #97, section "C_SET_TOPK_REG" (route weights are the softmax over the selected logits); the backward is the chain
rule of both.  ``contract=True`` rounds to bf16 where the GPU path stores bf16 for its products."""

from __future__ import annotations

import numpy as np

from oracle.moe_oracle import bf16_rne, silu


def _sigmoid(z):
    z = np.asarray(z, np.float64)
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def shared_fc1(x, ws1):
    """(act, h_pre): act = silu(g) * u of [g | u] = x @ ws1, ws1 [H, 2 I_s]."""
    h = np.asarray(x, np.float64) @ np.asarray(ws1, np.float64)
    half = h.shape[1] // 2
    return silu(h[:, :half]) * h[:, half:], h


def shared_fc2(act, ws2, x=None, w_gate=None):
    """(y, y_shared, gate): y = gate * (act @ ws2); y_shared and gate are None for the ungated block."""
    ys = np.asarray(act, np.float64) @ np.asarray(ws2, np.float64)
    if w_gate is None:
        return ys, None, None
    gate = _sigmoid(np.asarray(x, np.float64) @ np.asarray(w_gate, np.float64))
    return gate[:, None] * ys, ys, gate


def shared_fc2_backward(dy, act, h_pre, ws2, y_shared=None, gate=None, contract=False):
    """(d_h, d_ws2, d_gate_logit); with ``contract`` gate * dy is rounded to bf16 for the two products."""
    dy = np.asarray(dy, np.float64)
    D, d_z = dy, None
    if gate is not None:
        gate = np.asarray(gate, np.float64)
        D = gate[:, None] * dy
        d_z = gate * (1.0 - gate) * np.sum(dy * np.asarray(y_shared, np.float64), axis=1)
    if contract:
        D = bf16_rne((dy.astype(np.float32) * (1 if gate is None else gate.astype(np.float32)[:, None]))
                     ).astype(np.float64)
    da = D @ np.asarray(ws2, np.float64).T
    h = np.asarray(h_pre, np.float64)
    half = h.shape[1] // 2
    g, u = h[:, :half], h[:, half:]
    s = _sigmoid(g)
    d_h = np.concatenate([da * u * s * (1.0 + g * (1.0 - s)), da * g * s], axis=1)
    return d_h, np.asarray(act, np.float64).T @ D, d_z


def shared_fc1_backward(d_h, x, ws1, d_gate_logit=None, w_gate=None):
    """(d_x, d_ws1, d_w_gate)."""
    d_h, x = np.asarray(d_h, np.float64), np.asarray(x, np.float64)
    d_x = d_h @ np.asarray(ws1, np.float64).T
    d_wg = None
    if w_gate is not None:
        d_z = np.asarray(d_gate_logit, np.float64)
        d_x = d_x + np.outer(d_z, np.asarray(w_gate, np.float64))
        d_wg = x.T @ d_z
    return d_x, x.T @ d_h, d_wg


def route_backward(x, w_router, ids, weights, d_weights, contract=False):
    """(d_x, d_w_router, d_logit_bias, d_logits [T, E]); slots of one token that name one expert add up, ids outside
    [0, E) reach nothing.  With ``contract`` d_logits is rounded to bf16 for d_w_router."""
    x, wr = np.asarray(x, np.float64), np.asarray(w_router, np.float64)
    w, dw = np.asarray(weights, np.float64), np.asarray(d_weights, np.float64)
    T, k = w.shape
    E = wr.shape[1]
    dl = w * (dw - np.sum(w * dw, axis=1, keepdims=True))
    d_logits = np.zeros((T, E))
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                d_logits[t, ids[t, j]] += dl[t, j]
    stored = bf16_rne(d_logits.astype(np.float32)).astype(np.float64) if contract else d_logits
    return d_logits @ wr.T, x.T @ stored, d_logits.sum(axis=0), d_logits


def grad_norm(grads):
    """2-norm of all elements of all arrays together."""
    return float(np.sqrt(sum(np.sum(np.asarray(g, np.float64) ** 2) for g in grads)))


def clip_coef(norm, max_norm):
    """min(1, max_norm / (norm + 1e-6)), not a number when the norm is none."""
    c = max_norm / (norm + 1e-6)
    return 1.0 if c >= 1.0 else c
