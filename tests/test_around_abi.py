"""Refusals of the calls around the layer at the C ABI: invalid arguments are named on the host before a GPU is touched
(CPU only)."""

import ctypes
import math

import pytest

from mixture_experts_ffn_05_amd import binding as B

ODD4, ODD16 = ctypes.c_void_p(0x1002), ctypes.c_void_p(0x1004)
QUINTIC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def lib():
    return B.load()


def _err(lib):
    return lib.moe_last_error().decode()


class Args:
    """Pointers of a call's tensors, each of its own 16 MiB and never dereferenced."""

    def __init__(self, given):
        self.given, self.n = given, 0

    def __call__(self, name):
        self.n += 1
        if name in self.given:
            v = self.given[name]
            return v if v is None or isinstance(v, ctypes.c_void_p) else ctypes.c_void_p(v)
        return ctypes.c_void_p(self.n << 24)

    def at(self, i):
        return i << 24


def balance(lib, T=16, E=10, k=2, coef=0.01, z=0.1, ws=1 << 20, **ptrs):
    p = Args(ptrs)
    return lib.moe_balance_loss(p("logits"), p("topk_ids"), p("token_mask"), T, E, k, coef, z, p("losses"),
                                p("counts"), p("tokens"), p("prob_sums"), p("lse"), p("workspace"), ws, None)


def test_balance_loss(lib):
    assert lib.moe_balance_loss_workspace_bytes(0, 4) == 0 and lib.moe_balance_loss_workspace_bytes(4, 1025) == 0
    need = lib.moe_balance_loss_workspace_bytes(16, 10)
    assert need > 0 and lib.moe_balance_loss_workspace_bytes(1 << 20, 256) >= need
    assert balance(lib, T=0) == 1 and "T must be >= 1" in _err(lib)
    assert balance(lib, E=0) == 1 and balance(lib, E=1025) == 2
    assert balance(lib, k=0) == 1 and balance(lib, k=33) == 2
    assert balance(lib, T=1 << 27, k=2) == 2 and "T*top_k" in _err(lib)
    for name, v in (("coef", math.inf), ("coef", math.nan), ("z", -math.inf)):
        assert balance(lib, **{name: v}) == 1 and "finite" in _err(lib)
    for name in ("logits", "topk_ids", "losses", "counts", "tokens", "prob_sums", "lse"):
        assert balance(lib, **{name: None}) == 1 and name in _err(lib), name
        assert balance(lib, **{name: ODD4}) == 1 and "4-byte" in _err(lib), name
    assert balance(lib, workspace=None) == 3 and balance(lib, ws=need - 1) == 3
    assert balance(lib, workspace=ODD16) == 1 and "16-byte" in _err(lib)
    assert balance(lib, lse=1 << 24) == 1 and "lse overlaps logits" in _err(lib)
    assert balance(lib, tokens=(3 << 24) + 8) == 1 and "overlaps token_mask" in _err(lib)


def route(lib, dt=1, T=16, H=64, E=10, k=2, coef=0.01, z=0.1, acc=0, ws=1 << 23, **ptrs):
    p = Args(ptrs)
    return lib.moe_route_balance_backward(
        dt, p("x"), p("w_router"), p("logits"), p("lse"), p("topk_ids"), p("topk_weights"), p("d_topk_weights"),
        p("token_mask"), p("counts"), p("tokens"), T, H, E, k, coef, z, acc, p("d_x"), p("d_w_router"),
        p("d_logit_bias"), p("workspace"), ws, None)


def test_route_balance_backward(lib):
    for bad in ((2, 1, 8, 8), (1, 0, 8, 8), (1, 1, 0, 8), (1, 1, 8, 0), (1, 1, 8, 1025), (1, 1, (1 << 18) + 8, 8)):
        assert lib.moe_route_balance_backward_workspace_bytes(*bad) == 0, bad
    need = lib.moe_route_balance_backward_workspace_bytes(1, 16, 64, 10)
    assert need >= 16 * 16 * 6
    assert route(lib, dt=3) == 1 and route(lib, T=0) == 1 and route(lib, H=60) == 2 and route(lib, E=1025) == 2
    assert route(lib, k=0) == 1 and route(lib, k=33) == 2 and route(lib, acc=2) == 1
    assert route(lib, coef=math.nan) == 1 and route(lib, z=math.inf) == 1
    assert route(lib, dt=0, T=1 << 20, H=1 << 18) == 2 and "one launch" in _err(lib)
    for name in ("x", "w_router", "d_x", "d_w_router"):
        assert route(lib, **{name: None}) == 1 and name in _err(lib)
        assert route(lib, **{name: ctypes.c_void_p(0x1008)}) == 1 and "16-byte" in _err(lib)
    for name in ("logits", "lse", "counts", "tokens", "topk_ids"):
        assert route(lib, **{name: None}) == 1 and name in _err(lib)
    for name in ("logits", "lse", "counts", "tokens", "topk_ids", "topk_weights", "d_topk_weights", "d_logit_bias"):
        assert route(lib, **{name: ODD4}) == 1 and "4-byte" in _err(lib), name
    assert route(lib, topk_weights=None) == 1 and "both" in _err(lib)
    assert route(lib, d_topk_weights=None) == 1 and "both" in _err(lib)
    assert route(lib, ws=need - 1) == 3 and route(lib, workspace=None) == 3
    assert route(lib, d_x=1 << 24) == 1 and "d_x overlaps x" in _err(lib)
    assert route(lib, d_logit_bias=9 << 24) == 1 and "overlaps counts" in _err(lib)


NORM = ["h", "y", "w_post", "gate", "w_pre"]


def norm(lib, dt=1, sdt=1, T=16, H=64, eps=1e-6, off=0.0, rs=1.0, bs=1.0, **ptrs):
    p = Args(ptrs)
    head = [p(n) for n in NORM]
    return lib.moe_norm_residual(dt, sdt, *head, T, H, eps, off, rs, bs, p("h_out"), p("x"), p("rstd_post"),
                                 p("rstd_pre"), None)


def test_norm_residual(lib):
    assert norm(lib, dt=2) == 1 and norm(lib, sdt=-1) == 1 and "stream_dt" in _err(lib)
    assert norm(lib, T=0) == 1 and norm(lib, T=1 << 28) == 2 and norm(lib, H=0) == 1 and norm(lib, H=60) == 2
    assert norm(lib, H=8200) == 2 and "8192" in _err(lib)
    assert norm(lib, eps=-1.0) == 1 and norm(lib, eps=math.nan) == 1
    for name in ("off", "rs", "bs"):
        assert norm(lib, **{name: math.inf}) == 1 and "finite" in _err(lib)
    assert norm(lib, y=None, w_post=None, gate=None, w_pre=None, h_out=None, x=None, rstd_post=None,
                rstd_pre=None) == 1 and "both" in _err(lib)
    assert norm(lib, h=None) == 1 and norm(lib, h_out=None) == 1 and norm(lib, x=None) == 1
    none = dict(y=None, w_post=None, gate=None, h_out=None, rstd_post=None)
    for name in ("w_post", "gate", "h_out"):
        assert norm(lib, **{k: v for k, v in none.items() if k != name}) == 1 and f"{name} must be NULL" in _err(lib)
    assert norm(lib, w_post=None) == 1 and "rstd_post must be NULL" in _err(lib)
    assert norm(lib, w_pre=None) == 1 and "x must be NULL" in _err(lib)
    assert norm(lib, w_pre=None, x=None) == 1 and "rstd_pre must be NULL" in _err(lib)
    for name in NORM + ["h_out", "x"]:
        assert norm(lib, **{name: ctypes.c_void_p(0x1008)}) == 1 and "16-byte" in _err(lib), name
    for name in ("rstd_post", "rstd_pre"):
        assert norm(lib, **{name: ODD4}) == 1 and "4-byte" in _err(lib), name
    assert norm(lib, h_out=(1 << 24) + 16) == 1 and "h_out overlaps h" in _err(lib)
    assert norm(lib, x=2 << 24) == 1 and "x overlaps y" in _err(lib)


def norm_bwd(lib, dt=1, sdt=1, T=16, H=64, off=0.0, rs=1.0, bs=1.0, ws=1 << 23, **ptrs):
    p = Args(ptrs)
    head = [p(n) for n in ("d_h_out", "d_x", "h_out", "rstd_pre", "w_pre", "y", "rstd_post", "w_post", "gate")]
    return lib.moe_norm_residual_backward(dt, sdt, *head, T, H, off, rs, bs, p("d_h"), p("d_y"), p("d_w_pre"),
                                          p("d_w_post"), p("d_gate"), p("workspace"), ws, None)


def test_norm_residual_backward(lib):
    assert lib.moe_norm_residual_backward_workspace_bytes(0, 64) == 0
    assert lib.moe_norm_residual_backward_workspace_bytes(4, 8200) == 0
    need = lib.moe_norm_residual_backward_workspace_bytes(16, 64)
    assert need >= 3 * 64 * 4
    assert norm_bwd(lib, dt=2) == 1 and norm_bwd(lib, sdt=5) == 1 and norm_bwd(lib, T=0) == 1
    assert norm_bwd(lib, H=12) == 2 and norm_bwd(lib, rs=math.nan) == 1
    pre_none = dict(d_x=None, rstd_pre=None, w_pre=None, d_w_pre=None)
    assert norm_bwd(lib, d_h_out=None, **pre_none) == 1 and "both" in _err(lib)
    for name in ("h_out", "rstd_pre", "w_pre", "d_w_pre", "rstd_post", "d_w_post", "d_gate", "d_h"):
        assert norm_bwd(lib, **{name: None}) == 1 and name in _err(lib), name
    assert norm_bwd(lib, y=None) == 1 and "y" in _err(lib)
    for name in ("rstd_pre", "w_pre", "d_w_pre"):
        assert norm_bwd(lib, **{k: v for k, v in pre_none.items() if k != name}) == 1, name
        assert f"{name} must be NULL" in _err(lib), name
    branch_none = dict(d_y=None, w_post=None, rstd_post=None, gate=None, y=None, d_w_post=None, d_gate=None)
    for name in ("w_post", "rstd_post", "gate", "y", "d_w_post", "d_gate"):
        assert norm_bwd(lib, **{k: v for k, v in branch_none.items() if k != name}) == 1, name
        assert f"{name} must be NULL" in _err(lib), name
    for name in ("d_h_out", "d_x", "h_out", "w_pre", "y", "w_post", "gate", "d_h", "d_y", "d_w_pre"):
        assert norm_bwd(lib, **{name: ctypes.c_void_p(0x1008)}) == 1 and "16-byte" in _err(lib), name
    assert norm_bwd(lib, ws=need - 1) == 3 and norm_bwd(lib, workspace=None) == 3
    assert norm_bwd(lib, d_h=(1 << 24) + 16) == 1 and "d_h overlaps d_h_out" in _err(lib)
    assert norm_bwd(lib, d_y=6 << 24) == 1 and "d_y overlaps y" in _err(lib)


def ortho(lib, dt=1, odt=1, mu=0.9, nesterov=1, batch=2, M=16, N=24, parts=1, steps=5, coefs=QUINTIC * 5, eps=1e-7,
          scale=1.0, keep=0.0, ws=1 << 23, **ptrs):
    p = Args(ptrs)
    c = None if coefs is None else (ctypes.c_float * max(len(coefs), 1))(*coefs)
    return lib.moe_orthogonal_update(dt, odt, p("grad"), p("momentum"), mu, nesterov, batch, M, N, parts, steps, c, eps,
                                     scale, keep, p("out"), p("workspace"), ws, None)


def test_orthogonal_update(lib):
    q = lib.moe_orthogonal_update_workspace_bytes
    for bad in ((2, 1, 1, 8, 8, 1, 0), (1, 2, 1, 8, 8, 1, 0), (1, 1, 0, 8, 8, 1, 0), (1, 1, 1, 0, 8, 1, 0),
                (1, 1, 1, 8, 0, 1, 0), (1, 1, 1, 8, 8, 0, 0), (1, 1, 1, 32769, 8, 1, 0), (1, 1, 1, 8, 32769, 1, 0),
                (1, 1, 65536, 8, 8, 1, 0), (1, 1, 40000, 8, 8, 2, 0)):
        assert q(*bad) == 0, bad
    need = q(1, 1, 2, 16, 24, 1, 1)
    assert need > 0
    for m, n in ((1, 1), (64, 2048), (65, 64), (129, 4096), (1000, 1001)):
        for out in (0, 1):
            assert q(1, out, 1, m, n, 1, 0) > 0 and q(0, out, 1, n, m, 1, 1) > 0, (m, n)
    assert ortho(lib, dt=2) == 1 and ortho(lib, odt=7) == 1 and "out_dt" in _err(lib)
    assert ortho(lib, batch=0) == 1 and ortho(lib, M=0) == 1 and ortho(lib, N=-1) == 1 and ortho(lib, parts=0) == 1
    assert ortho(lib, M=32769) == 2 and ortho(lib, batch=65536) == 2 and "65535" in _err(lib)
    assert ortho(lib, nesterov=2) == 1 and ortho(lib, steps=0) == 1 and ortho(lib, steps=17, coefs=(1, 0, 0) * 17) == 2
    assert ortho(lib, coefs=None) == 1 and ortho(lib, coefs=(math.nan,) * 15) == 1 and "coefs" in _err(lib)
    for name in ("mu", "scale", "keep"):
        assert ortho(lib, **{name: math.inf}) == 1 and name in _err(lib)
    for eps in (0.0, -1.0, 0.9e-12, math.inf, math.nan):
        assert ortho(lib, eps=eps) == 1 and "eps" in _err(lib)
    assert ortho(lib, steps=2, coefs=(100.0, 0.0, 0.0) * 2) == 2 and "beyond 64" in _err(lib)
    assert ortho(lib, grad=None) == 1 and ortho(lib, out=None) == 1
    assert ortho(lib, grad=ctypes.c_void_p(0x1001)) == 1 and "grad must be 2-byte" in _err(lib)
    assert ortho(lib, momentum=ODD4) == 1 and ortho(lib, dt=0, grad=ODD4) == 1
    assert ortho(lib, odt=0, out=ODD4) == 1 and "out must be 4-byte" in _err(lib)
    assert ortho(lib, ws=need - 1) == 3 and ortho(lib, workspace=None) == 3 and ortho(lib, workspace=ODD16) == 1
    assert ortho(lib, out=1 << 24) == 1 and "out overlaps grad" in _err(lib)
    assert ortho(lib, momentum=(1 << 24) + 64) == 1 and "momentum overlaps grad" in _err(lib)


def test_stages(lib):
    for call, stage in (("moe_balance_loss", "router_topk"), ("moe_route_balance_backward", "backward:router_topk"),
                        ("moe_norm_residual", "residual_setup"),
                        ("moe_norm_residual_backward", "backward:residual_setup"),
                        ("moe_orthogonal_update", "backward:other")):
        assert B.moe_call_stage(call) == stage
