"""Refusals of the training calls at the C ABI: invalid arguments are named on the host before a GPU is touched (CPU
only), also in the library's copy built with host-side sanitizers."""

import ctypes
import os
import subprocess
import sys

import pytest

from mixture_experts_ffn_05_amd import binding as B

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every case fails validation first
ODD = ctypes.c_void_p(0x1008)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    return B.load()


def _err(lib):
    return lib.moe_last_error().decode()


def test_workspace_sizes(lib):
    need = lib.moe_shared_train_workspace_bytes(1, 100, 64, 72)
    assert need >= 100 * 64 * 2
    assert lib.moe_shared_train_workspace_bytes(0, 100, 64, 72) >= 100 * 64 * 4
    for bad in ((2, 1, 8, 8), (1, 0, 8, 8), (1, 1, 0, 8), (1, 1, 8, 0), (1, 1, 8, (1 << 18) + 8)):
        assert lib.moe_shared_train_workspace_bytes(*bad) == 0, bad
    assert lib.moe_route_backward_workspace_bytes(1, 100, 64, 10, 2) > 0
    for bad in ((2, 1, 8, 8, 1), (1, 0, 8, 8, 1), (1, 1, 0, 8, 1), (1, 1, 8, 0, 1), (1, 1, 8, 1025, 1), (1, 1, 8, 8, 0),
                (1, 1, 8, 8, 33)):
        assert lib.moe_route_backward_workspace_bytes(*bad) == 0, bad
    assert lib.moe_grad_norm_workspace_bytes(0) == 0 and lib.moe_grad_norm_workspace_bytes(-3) == 0
    assert lib.moe_grad_norm_workspace_bytes(1) > 0
    assert lib.moe_grad_norm_workspace_bytes(1000) > lib.moe_grad_norm_workspace_bytes(1)


SHARED_CALLS = {
    "moe_shared_fc1_save": dict(tensors=["x", "ws1"], after=["act", "h_pre"], flag=False),
    "moe_shared_fc2_save": dict(tensors=["act", "ws2", "x", "w_gate"], after=["y", "y_shared", "gate"], flag=True),
    "moe_shared_fc2_backward": dict(tensors=["dy", "act", "h_pre", "ws2", "y_shared", "gate"],
                                    after=["d_h", "d_ws2", "d_gate_logit"], flag=False),
    "moe_shared_fc1_backward": dict(tensors=["d_h", "x", "ws1", "d_gate_logit", "w_gate"],
                                    after=["d_x", "d_ws1", "d_w_gate"], flag=True),
}
GATE = {"w_gate", "y_shared", "gate", "d_gate_logit", "d_w_gate"}
KEY = {"moe_shared_fc2_save": "w_gate", "moe_shared_fc2_backward": "gate", "moe_shared_fc1_backward": "w_gate"}


def _shared(lib, fn, dt=1, wl=0, T=16, H=64, I_s=72, acc=0, ws=FAKE, ws_bytes=1 << 30, **ptrs):
    c = SHARED_CALLS[fn]
    p = lambda n: ptrs.get(n, FAKE)   # noqa: E731
    args = [dt, wl, *[p(n) for n in c["tensors"]], T, H, I_s]
    args += [acc] if c["flag"] else []
    return getattr(lib, fn)(*args, *[p(n) for n in c["after"]], ws, ws_bytes, None)


@pytest.mark.parametrize("fn", SHARED_CALLS)
def test_shared_calls(lib, fn):
    c = SHARED_CALLS[fn]
    assert _shared(lib, fn, dt=2) == 1 and "dt" in _err(lib)
    assert _shared(lib, fn, wl=2) == 1 and "weight layout" in _err(lib)
    assert _shared(lib, fn, T=0) == 1 and "T must be >= 1" in _err(lib)
    assert _shared(lib, fn, T=1 << 28) == 2 and "T must be <" in _err(lib)
    assert _shared(lib, fn, H=0) == 1 and _shared(lib, fn, I_s=-8) == 1
    assert _shared(lib, fn, H=68) == 2 and "H must be a multiple of 8" in _err(lib)
    assert _shared(lib, fn, I_s=4) == 2 and "I_s must be a multiple of 8" in _err(lib)
    assert _shared(lib, fn, H=(1 << 18) + 8) == 2 and _shared(lib, fn, I_s=(1 << 18) + 8) == 2
    assert _shared(lib, fn, H=1 << 14, I_s=1 << 14) == 2 and "H * I_s" in _err(lib)
    for name in c["tensors"] + c["after"]:
        assert _shared(lib, fn, **{name: ODD}) == 1 and name in _err(lib) and "16-byte" in _err(lib), name
        if name != KEY.get(fn):
            assert _shared(lib, fn, **{name: None}) == 1 and name in _err(lib), name
    if fn in KEY:   # ungated: nothing that belongs to the gate may be given
        gate = [n for n in c["tensors"] + c["after"] if n in GATE]
        for name in gate:
            if name != KEY[fn]:
                none = {n: None for n in gate if n != name}
                assert _shared(lib, fn, **none) == 1 and f"{name} must be NULL" in _err(lib), name
    if c["flag"]:
        assert _shared(lib, fn, acc=2) == 1 and "accumulate" in _err(lib)
    need = lib.moe_shared_train_workspace_bytes(1, 16, 64, 72)
    assert _shared(lib, fn, ws_bytes=need - 1) == 3 and "workspace needs" in _err(lib)
    assert _shared(lib, fn, ws=None) == 3
    assert _shared(lib, fn, ws=ODD) == 1 and "workspace" in _err(lib)


def test_route_backward(lib):
    names = ["x", "w_router", "topk_ids", "topk_weights", "d_topk_weights"]

    def call(dt=1, T=16, H=64, E=10, k=2, acc=0, ws=FAKE, ws_bytes=1 << 30, **ptrs):
        p = lambda n: ptrs.get(n, FAKE)   # noqa: E731
        return lib.moe_route_backward(dt, *[p(n) for n in names], T, H, E, k, acc, p("d_x"), p("d_w_router"),
                                      p("d_logit_bias"), ws, ws_bytes, None)

    assert call(dt=5) == 1
    assert call(T=0) == 1 and call(H=0) == 1 and call(E=0) == 1
    assert call(k=0) == 1 and "top_k must be positive" in _err(lib)
    assert call(k=33) == 2 and call(E=1025) == 2 and call(H=60) == 2 and call(H=(1 << 18) + 8) == 2
    assert call(T=1 << 27, k=2) == 2 and "T*top_k" in _err(lib)
    assert call(acc=-1) == 1 and "accumulate" in _err(lib)
    for n in names + ["d_x", "d_w_router"]:
        assert call(**{n: None}) == 1 and n in _err(lib), n
    for n in ("x", "w_router", "d_x", "d_w_router"):
        assert call(**{n: ODD}) == 1 and "16-byte" in _err(lib), n
    for n in ("topk_ids", "topk_weights", "d_topk_weights", "d_logit_bias"):
        assert call(**{n: ctypes.c_void_p(0x1002)}) == 1 and "4-byte" in _err(lib), n
    need = lib.moe_route_backward_workspace_bytes(1, 16, 64, 10, 2)
    assert call(ws_bytes=need - 1) == 3 and call(ws=None) == 3 and call(ws=ODD) == 1


def _grads(n, ptrs=None, numel=None, dts=None):
    vp = ctypes.c_void_p * max(n, 1)
    return (vp(*(ptrs or [0x1000 + 0x1000 * i for i in range(n)])),
            (ctypes.c_int64 * max(n, 1))(*(numel or [16] * n)), (ctypes.c_int32 * max(n, 1))(*(dts or [1] * n)))


def test_grad_norm(lib):
    def call(n=2, ptrs=None, numel=None, dts=None, norm=FAKE, sq=None, ws=FAKE, wsb=1 << 20, lists=None):
        g, m, d = lists or _grads(n, ptrs, numel, dts)
        return lib.moe_grad_norm(n, g, m, d, norm, sq, ws, wsb, None)

    assert call(n=0) == 1 and "n must be >= 1" in _err(lib)
    assert call(n=-1, lists=_grads(1)) == 1
    g, m, d = _grads(2)
    assert call(lists=(None, m, d)) == 1 and call(lists=(g, None, d)) == 1 and call(lists=(g, m, None)) == 1
    assert call(dts=[1, 2]) == 1 and "dts[1]" in _err(lib)
    assert call(numel=[3, -1]) == 1 and "numel[1]" in _err(lib)
    assert call(numel=[1 << 42, 1 << 42]) == 2 and "2^43" in _err(lib)
    assert call(ptrs=[0x1000, 0]) == 1 and "grads[1] must not be NULL" in _err(lib)
    assert call(ptrs=[0x1001, 0x2000]) == 1 and "aligned" in _err(lib)
    assert call(ptrs=[0x1002, 0x2000], dts=[0, 0]) == 1 and "grads[0]" in _err(lib)
    assert call(norm=None) == 1 and call(norm=ctypes.c_void_p(0x1002)) == 1
    assert call(sq=ctypes.c_void_p(0x1004)) == 1 and "sum_sq" in _err(lib)
    assert call(ws=None) == 3 and call(wsb=lib.moe_grad_norm_workspace_bytes(2) - 1) == 3
    assert call(ws=ctypes.c_void_p(0x1004)) == 1


def test_grad_clip(lib):
    def call(n=2, ptrs=None, outs=None, numel=None, dts=None, norm=FAKE, max_norm=1.0, coef=None, out_arr=True):
        g, m, d = _grads(n, ptrs, numel, dts)
        o = (ctypes.c_void_p * max(n, 1))(*(outs or [0x100000 + 0x1000 * i for i in range(n)])) if out_arr else None
        return lib.moe_grad_clip(n, g, o, m, d, norm, max_norm, coef, None)

    assert call(n=0) == 1
    assert call(out_arr=False) == 1 and "outs" in _err(lib)
    assert call(outs=[0x100000, 0]) == 1 and "outs[1]" in _err(lib)
    assert call(outs=[0x100001, 0x200000]) == 1 and "aligned" in _err(lib)
    for m in (float("nan"), float("inf"), -1.0):
        assert call(max_norm=m) == 1 and "max_norm" in _err(lib), m
    assert call(norm=None) == 1 and call(coef=ctypes.c_void_p(0x1002)) == 1
    # 16 bf16 elements are 32 bytes
    assert call(outs=[0x100000, 0x10001e]) == 1 and "overlaps" in _err(lib)          # two outputs
    assert call(outs=[0x2002, 0x100000]) == 1 and "overlaps" in _err(lib)            # an output and another's input
    assert call(outs=[0x1002, 0x100000]) == 1 and "overlaps" in _err(lib)            # its own input, shifted
    assert call(ptrs=[0x1000, 0x1000], outs=[0x1000, 0x1000]) == 1 and "overlaps" in _err(lib)   # one tensor twice
    assert call(ptrs=[0x1000, 0x1000], outs=[0x1000, 0x9000]) == 1 and "overlaps" in _err(lib)
    # a long tensor that starts first reaches past a short one
    assert call(numel=[10000, 16], outs=[0x100000, 0x100000 + 16000]) == 1 and "overlaps" in _err(lib)


def _sizes(fn, e, T, H, I_s):
    return {"x": e * T * H, "ws1": 2 * e * H * I_s, "act": e * T * I_s, "h_pre": 2 * e * T * I_s, "ws2": e * I_s * H,
            "w_gate": e * H, "y": 4 * T * H, "y_shared": 4 * T * H, "gate": 4 * T, "dy": 4 * T * H,
            "d_h": 2 * e * T * I_s, "d_ws2": e * I_s * H, "d_gate_logit": 4 * T, "d_x": 4 * T * H,
            "d_ws1": 2 * e * H * I_s, "d_w_gate": e * H}


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("fn", SHARED_CALLS)
def test_shared_calls_refuse_overlaps(lib, fn, dt):
    T, H, I_s = 16, 64, 72
    c, size = SHARED_CALLS[fn], _sizes(fn, 4 if dt == 0 else 2, T, H, I_s)
    names = c["tensors"] + c["after"]
    place = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}
    work = 0x100000 * (len(names) + 1)
    for out in c["after"]:   # each output laid over each other argument's last 16 bytes
        for other in names:
            if other == out:
                continue
            end = place[other] + (size[other] + 15) // 16 * 16 - 16
            got = _shared(lib, fn, dt=dt, ws=work, **{**place, out: end})
            assert got == 1 and "overlaps" in _err(lib) and out in _err(lib) and other in _err(lib), (out, other)
        assert _shared(lib, fn, dt=dt, ws=work, **{**place, out: work}) == 1 and "workspace overlaps" in _err(lib)
    for other in names:
        assert _shared(lib, fn, dt=dt, ws=place[other], **place) == 1 and "overlaps" in _err(lib), other


def test_route_backward_refuses_overlaps(lib):
    names = ["x", "w_router", "topk_ids", "topk_weights", "d_topk_weights"]
    outs = ["d_x", "d_w_router", "d_logit_bias"]
    size = {"x": 2 * 16 * 64, "w_router": 2 * 64 * 10, "topk_ids": 128, "topk_weights": 128, "d_topk_weights": 128,
            "d_x": 4 * 16 * 64, "d_w_router": 2 * 64 * 10, "d_logit_bias": 40}
    place = {n: 0x100000 * (i + 1) for i, n in enumerate(names + outs)}

    def call(ws=0x2000000, **ptrs):
        p = {**place, **ptrs}
        return lib.moe_route_backward(1, *[p[n] for n in names], 16, 64, 10, 2, 0, *[p[n] for n in outs], ws, 1 << 30,
                                      None)

    for out in outs:
        for other in names + outs:
            if other != out:
                end = place[other] + (size[other] + 15) // 16 * 16 - 16
                assert call(**{out: end}) == 1 and "overlaps" in _err(lib) and out in _err(lib), (out, other)
        assert call(ws=place[out]) == 1 and f"workspace overlaps {out}" in _err(lib)


def test_grad_calls_refuse_overlapping_scalars(lib):
    g, m, d = _grads(2)                     # 32 bytes each at 0x1000 and 0x2000
    o = (ctypes.c_void_p * 2)(0x100000, 0x200000)
    def norm(nm=0x8000000, sq=0x9000000, ws=0x10000000):
        return lib.moe_grad_norm(2, g, m, d, nm, sq, ws, 1 << 20, None)

    assert norm(sq=0x8000000) == 1 and "sum_sq overlaps norm" in _err(lib)
    assert norm(nm=0x8000004, sq=0x8000000) == 1
    assert norm(nm=0x10000010) == 1 and "workspace overlaps norm" in _err(lib)
    assert norm(nm=0x101c) == 1 and "norm overlaps grads[0]" in _err(lib)
    assert norm(sq=0x2018) == 1 and "sum_sq overlaps grads[1]" in _err(lib)
    assert norm(ws=0x0ff0) == 1 and "workspace overlaps grads[0]" in _err(lib)
    clip = lambda nm, coef, outs=o: lib.moe_grad_clip(2, g, outs, m, d, nm, 1.0, coef, None)   # noqa: E731
    assert clip(0x8000, 0x8000) == 1 and "overlaps" in _err(lib)
    assert clip(0x100010, None) == 1 and "norm overlaps" in _err(lib)
    assert clip(0x8000, 0x200000) == 1 and "overlaps" in _err(lib)
    assert clip(0x8000, 0x1010) == 1 and "coef overlaps" in _err(lib)
    assert clip(0x8000, 0x1010, g) == 1 and "coef overlaps" in _err(lib)   # in place


def test_train_tiles(lib):
    splits = (ctypes.c_int32 * 2)(7, 7)
    for call in range(4):
        assert lib.moe_shared_train_tiles(0, call, 0, 16, 64, 72, splits) == B.MOE_DENSE_F32
        assert list(splits) == [1, 1]
        splits[0] = splits[1] = 7
    for bad in ((2, 0, 0, 16, 64, 72), (0, -1, 0, 16, 64, 72), (0, 4, 0, 16, 64, 72), (0, 0, 2, 16, 64, 72),
                (0, 0, 0, 0, 64, 72), (0, 0, 0, 16, 60, 72), (0, 0, 0, 16, 64, 4), (0, 0, 0, 1 << 28, 64, 72)):
        assert lib.moe_shared_train_tiles(*bad, splits) == -1, bad
    assert lib.moe_shared_train_tiles(0, 0, 0, 16, 64, 72, None) == -1
    assert list(splits) == [7, 7]


def test_layer_calls_refuse_buffers_of_another_layer():
    """A layer's gradient list holds what its buffers were made for: a shared expert or a gate or a bias that the call
    leaves out would put memory that nobody wrote into the norm."""
    from types import SimpleNamespace as NS
    shared = ("ws1", "ws2", "w_gate")
    plain = ("ws1", "ws2", None)
    for train, sh, bias in ((NS(I_s=64, gated=True, d_logit_bias=None), None, None),
                            (NS(I_s=0, gated=False, d_logit_bias=None), shared, None),
                            (NS(I_s=64, gated=True, d_logit_bias=None), plain, None),
                            (NS(I_s=64, gated=False, d_logit_bias=None), shared, None),
                            (NS(I_s=0, gated=False, d_logit_bias=None), None, "bias"),
                            (NS(I_s=0, gated=False, d_logit_bias="d"), None, None)):
        with pytest.raises(ValueError, match="were made for"):
            B.moe_layer_train_forward(None, None, bias, None, None, 2, sh, None, train)
        if (train.d_logit_bias is None) == (bias is None):
            with pytest.raises(ValueError, match="were made for"):
                B.moe_layer_backward(None, None, None, None, None, sh, None, train)


def test_refusals_under_host_sanitizers():
    from mixture_experts_ffn_05_amd import build
    if os.environ.get("LIBMOE_LIBRARY"):
        pytest.skip("already the sanitized copy")
    lib = build.build_sanitized()
    preload = build.asan_runtime()
    if os.environ.get("LD_PRELOAD"):
        preload += ":" + os.environ["LD_PRELOAD"]
    env = {**os.environ, "LIBMOE_LIBRARY": lib, "LD_PRELOAD": preload,
           "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1", "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"}
    res = subprocess.run([sys.executable, "-m", "pytest", os.path.join("tests", "test_train_abi.py"), "-q", "-s",
                          "-p", "no:cacheprovider"], env=env, cwd=ROOT, capture_output=True, text=True, timeout=1200)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-4000:]
    assert "Sanitizer" not in out, out[-4000:]
    assert " passed" in res.stdout
