"""Thin ctypes binding of libmoe's C ABI (include/libmoe.h).

Each function here has the name of the C call it wraps and only marshals
arguments: it checks devices, dtypes, shapes and contiguity of torch tensors,
passes their device pointers and the current HIP stream, and raises MoEError
on a non-zero status.  Every step of the layer runs in libmoe's HIP kernels;
there is no fallback of any kind.  If libmoe.so has not been built, load()
raises.
"""

from __future__ import annotations

import ctypes
import os
import re
from typing import NamedTuple

import torch

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libmoe.so")
HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "libmoe.h")

MOE_F32, MOE_BF16 = 0, 1
MOE_W_KN, MOE_W_NK = 0, 1   # expert weights as [K, N] (x @ W) or [N, K] (torch.nn.Linear)
MOE_OK = 0

_lib = None


def moe_call_stage(call: str, gated: bool = False) -> str:
    """Stage label of a libmoe call (the name of the roctx range it opens)."""
    return load().moe_call_stage(call.encode(), int(bool(gated))).decode()


class MoEError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} [{status}]")
        self.status = status


_c_int, _c_size, _vp = ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p
_c_float = ctypes.c_float

_SIGNATURES = {
    "moe_status_name": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_version": (ctypes.c_int, []),
    "moe_call_stage": (ctypes.c_char_p, [ctypes.c_char_p, _c_int]),
    "moe_route": (_c_int, [_c_int, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_size,
                           _vp]),
    "moe_route_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "moe_build_scatter_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int]),
    "moe_route_and_scatter": (_c_int, [_c_int, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp,
                                       _vp, _vp, _vp, _vp, _c_size, _vp]),
    "moe_route_and_scatter_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "moe_route_and_scatter_noalloc": (_c_int, [_c_int, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp,
                                               _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_route_and_scatter_noalloc_max_bytes": (_c_size, []),
    "moe_build_scatter": (_c_int, [_c_int, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp,
                                   _vp, _c_size, _vp]),
    "moe_grouped_swiglu_fc1": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp]),
    "moe_grouped_fc2": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp]),
    "moe_gather_combine": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp]),
    "moe_shared_expert_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int]),
    "moe_shared_expert": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp,
                                   _c_size, _vp]),
    "moe_grouped_swiglu_fc1_mx8": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp]),
    "moe_grouped_fc2_mx8": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp]),
    "moe_shared_expert_mx8": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp,
                                       _c_size, _vp]),
    "moe_grouped_swiglu_fc1_and_shared_mx8": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp,
                                                       _vp, _vp, _vp, _c_int, _c_int, _vp, _vp]),
    "moe_grouped_fc2_and_shared_mx8": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp,
                                                _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _c_size,
                                                _vp]),
    "moe_and_shared_launches": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "moe_grouped_gemm_tile": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "moe_grouped_swiglu_fc1_and_shared": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                                   _vp, _vp, _vp, _c_int, _c_int, _vp, _vp]),
    "moe_grouped_fc2_and_shared": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp,
                                            _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _c_size, _vp]),
    "moe_grouped_swiglu_fc1_gather": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                               _c_int, _vp, _vp]),
    "moe_grouped_swiglu_fc1_and_shared_gather": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_int,
                                                          _c_int, _c_int, _vp, _vp, _c_int, _c_int, _vp, _vp]),
    "moe_grouped_swiglu_fc1_save": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp,
                                             _vp, _vp]),
    "moe_scatter_grad": (_c_int, [_c_int, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "moe_grouped_fc2_backward": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                          _vp, _vp, _vp]),
    "moe_grouped_fc1_backward_workspace_bytes": (_c_size, [_c_int, _c_int]),
    "moe_grouped_fc1_backward": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp,
                                          _c_int, _c_int, _c_int, _vp, _vp, _vp, _c_size, _vp]),
    "moe_shared_train_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "moe_shared_train_tiles": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _vp]),
    "moe_shared_fc1_save": (_c_int, [_c_int, _c_int, _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _c_size, _vp]),
    "moe_shared_fc2_save": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp,
                                     _vp, _vp, _c_size, _vp]),
    "moe_shared_fc2_backward": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp,
                                         _vp, _vp, _vp, _c_size, _vp]),
    "moe_shared_fc1_backward": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                         _vp, _vp, _vp, _vp, _c_size, _vp]),
    "moe_route_backward_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "moe_route_backward": (_c_int, [_c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp,
                                    _vp, _vp, _vp, _c_size, _vp]),
    "moe_balance_loss_workspace_bytes": (_c_size, [_c_int, _c_int]),
    "moe_balance_loss": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _c_float, _c_float, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _c_size, _vp]),
    "moe_route_balance_backward_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "moe_route_balance_backward": (_c_int, [_c_int, *[_vp] * 10, _c_int, _c_int, _c_int, _c_int, _c_float, _c_float,
                                            _c_int, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "moe_norm_residual": (_c_int, [_c_int, _c_int, *[_vp] * 5, _c_int, _c_int, *[_c_float] * 4, _vp, _vp, _vp, _vp,
                                   _vp]),
    "moe_norm_residual_backward_workspace_bytes": (_c_size, [_c_int, _c_int]),
    "moe_norm_residual_backward": (_c_int, [_c_int, _c_int, *[_vp] * 9, _c_int, _c_int, *[_c_float] * 3, *[_vp] * 6,
                                            _c_size, _vp]),
    "moe_orthogonal_update_workspace_bytes": (_c_size, [_c_int] * 7),
    "moe_orthogonal_update": (_c_int, [_c_int, _c_int, _vp, _vp, _c_float, *[_c_int] * 6, _vp, *[_c_float] * 3, _vp,
                                       _vp, _c_size, _vp]),
    "moe_grad_norm_workspace_bytes": (_c_size, [_c_int]),
    "moe_grad_norm": (_c_int, [_c_int, _vp, _vp, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "moe_grad_clip": (_c_int, [_c_int, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp]),
}


def header_functions() -> list[str]:
    """Names of the functions include/libmoe.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libmoe.so (once) and declare its signatures.  Raises if it is missing.
    LIBMOE_LIBRARY in the environment names another build of the library (the
    host-sanitized copy the ABI tests run against)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or os.environ.get("LIBMOE_LIBRARY") or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libmoe.so not found at {p}: build it with "
                           "`python -m mixture_experts_ffn_05_amd.build` (there is no fallback path)")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != MOE_OK:
        lib = load()
        raise MoEError(status, f"{lib.moe_status_name(status).decode()}: {lib.moe_last_error().decode()}")


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.float32:
        return MOE_F32
    raise TypeError(f"unsupported dtype {t.dtype}: libmoe takes float32 or bfloat16")


def _ptr(t, name, dtype=None, shape=None, device=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    return t.data_ptr()


# The current stream's handle without a Stream object around it (1.5 us less per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _call_on(device, fn, *args):
    """fn(*args) with the tensors' device current (kernels launch on the current device)."""
    if torch.cuda.current_device() == device.index:
        return _check(fn(*args))
    with torch.cuda.device(device):
        _check(fn(*args))


def moe_route_workspace_bytes(dtype, T, H, E) -> int:
    dt = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(load().moe_route_workspace_bytes(dt, int(T), int(H), int(E)))


def moe_route(x, w_router, logit_bias, top_k, topk_ids, topk_weights, logits, workspace, stream=None):
    lib = load()
    T, H = x.shape
    E = w_router.shape[1]
    dev = x.device
    ws_ptr = _ptr(workspace, "workspace", torch.uint8, None, dev) if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    args = (_dt(x), _ptr(x, "x"), _ptr(w_router, "w_router", x.dtype, (H, E), dev),
            _ptr(logit_bias, "logit_bias", torch.float32, (E,), dev), T, H, E, int(top_k),
            _ptr(topk_ids, "topk_ids", torch.int32, (T, top_k), dev),
            _ptr(topk_weights, "topk_weights", torch.float32, (T, top_k), dev),
            _ptr(logits, "logits", torch.float32, (T, E), dev), ws_ptr, ws_bytes, _stream(stream, dev))
    _call_on(dev, lib.moe_route, *args)


def moe_build_scatter_workspace_bytes(T, top_k, E) -> int:
    return int(load().moe_build_scatter_workspace_bytes(int(T), int(top_k), int(E)))


def moe_build_scatter(x, topk_ids, num_experts, scatter_index, row_token, expert_offsets, status_words,
                      x_scattered, workspace, stream=None):
    lib = load()
    T, H = x.shape
    k = topk_ids.shape[1]
    E = int(num_experts)
    dev = x.device
    args = (_dt(x), _ptr(x, "x"), _ptr(topk_ids, "topk_ids", torch.int32, (T, k), dev), T, H, E, k,
            _ptr(scatter_index, "scatter_index", torch.int32, (T, k), dev),
            _ptr(row_token, "row_token", torch.int32, (T * k,), dev),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(status_words, "status_words", torch.int32, (2,), dev),
            _ptr(x_scattered, "x_scattered", x.dtype, (T * k, H), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_build_scatter, *args)


def moe_route_and_scatter_workspace_bytes(dtype, T, H, E, top_k) -> int:
    dt = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(load().moe_route_and_scatter_workspace_bytes(dt, int(T), int(H), int(E), int(top_k)))


def moe_route_and_scatter(x, w_router, logit_bias, top_k, topk_ids, topk_weights, logits, scatter_index, row_token,
                          expert_offsets, status_words, x_scattered, workspace, stream=None):
    lib = load()
    T, H = x.shape
    E = w_router.shape[1]
    k = int(top_k)
    dev = x.device
    args = (_dt(x), _ptr(x, "x"), _ptr(w_router, "w_router", x.dtype, (H, E), dev),
            _ptr(logit_bias, "logit_bias", torch.float32, (E,), dev), T, H, E, k,
            _ptr(topk_ids, "topk_ids", torch.int32, (T, k), dev),
            _ptr(topk_weights, "topk_weights", torch.float32, (T, k), dev),
            _ptr(logits, "logits", torch.float32, (T, E), dev),
            _ptr(scatter_index, "scatter_index", torch.int32, (T, k), dev),
            _ptr(row_token, "row_token", torch.int32, (T * k,), dev),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(status_words, "status_words", torch.int32, (2,), dev),
            _ptr(x_scattered, "x_scattered", x.dtype, (T * k, H), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_route_and_scatter, *args)


def moe_route_and_scatter_noalloc_max_bytes() -> int:
    return int(load().moe_route_and_scatter_noalloc_max_bytes())


def moe_route_and_scatter_noalloc(x, w_router, logit_bias, top_k, topk_ids, topk_weights, logits, scatter_index,
                                  row_token, expert_offsets, status_words, x_scattered, stream=None):
    lib = load()
    T, H = x.shape
    E = w_router.shape[1]
    k = int(top_k)
    dev = x.device
    args = (_dt(x), _ptr(x, "x"), _ptr(w_router, "w_router", x.dtype, (H, E), dev),
            _ptr(logit_bias, "logit_bias", torch.float32, (E,), dev), T, H, E, k,
            _ptr(topk_ids, "topk_ids", torch.int32, (T, k), dev),
            _ptr(topk_weights, "topk_weights", torch.float32, (T, k), dev),
            _ptr(logits, "logits", torch.float32, (T, E), dev),
            _ptr(scatter_index, "scatter_index", torch.int32, (T, k), dev),
            _ptr(row_token, "row_token", torch.int32, (T * k,), dev),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(status_words, "status_words", torch.int32, (2,), dev),
            _ptr(x_scattered, "x_scattered", x.dtype, (T * k, H), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_route_and_scatter_noalloc, *args)


def _fc1_sizes(w1, layout):
    """(E, H, I) of a stacked fc1 weight in the given layout."""
    if layout == MOE_W_NK:
        E, I2, H = w1.shape
    else:
        E, H, I2 = w1.shape
    return E, H, I2 // 2


def moe_grouped_swiglu_fc1(x_scattered, expert_offsets, w1, act, stream=None, layout=MOE_W_KN):
    lib = load()
    R, H = x_scattered.shape
    E, _, I = _fc1_sizes(w1, layout)
    dev = x_scattered.device
    wshape = (E, 2 * I, H) if layout == MOE_W_NK else (E, H, 2 * I)
    args = (_dt(x_scattered), int(layout), _ptr(x_scattered, "x_scattered"),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w1, "w1", x_scattered.dtype, wshape, dev), R, H, E, I,
            _ptr(act, "act", x_scattered.dtype, (R, I), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_swiglu_fc1, *args)


def moe_grouped_swiglu_fc1_gather(x, row_token, expert_offsets, w1, act, stream=None, layout=MOE_W_KN):
    """moe_grouped_swiglu_fc1 reading routed row r as x[row_token[r]] (no x_scattered)."""
    lib = load()
    T, H = x.shape
    R = row_token.shape[0]
    E, _, I = _fc1_sizes(w1, layout)
    dev = x.device
    wshape = (E, 2 * I, H) if layout == MOE_W_NK else (E, H, 2 * I)
    args = (_dt(x), int(layout), _ptr(x, "x"), _ptr(row_token, "row_token", torch.int32, (R,), dev),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w1, "w1", x.dtype, wshape, dev), T, R, H, E, I,
            _ptr(act, "act", x.dtype, (R, I), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_swiglu_fc1_gather, *args)


def moe_grouped_fc2(act, expert_offsets, w2, y_rows, stream=None, layout=MOE_W_KN):
    lib = load()
    R, I = act.shape
    E = w2.shape[0]
    H = w2.shape[1] if layout == MOE_W_NK else w2.shape[2]
    dev = act.device
    wshape = (E, H, I) if layout == MOE_W_NK else (E, I, H)
    args = (_dt(act), int(layout), _ptr(act, "act"),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w2, "w2", act.dtype, wshape, dev), R, I, E, H,
            _ptr(y_rows, "y_rows", torch.float32, (R, H), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_fc2, *args)


def moe_gather_combine(y_rows, scatter_index, topk_weights, y, accumulate=False, stream=None):
    lib = load()
    T, k = scatter_index.shape
    H = y.shape[1]
    dev = y.device
    args = (_ptr(y_rows, "y_rows", torch.float32, None, dev),
            _ptr(scatter_index, "scatter_index", torch.int32, (T, k), dev),
            _ptr(topk_weights, "topk_weights", torch.float32, (T, k), dev), T, H, k, int(bool(accumulate)),
            _ptr(y, "y", torch.float32, (T, H), dev), _stream(stream, dev))
    if y_rows.dim() != 2 or y_rows.shape[1] != H:
        raise ValueError("y_rows must be [R, H]")
    _call_on(dev, lib.moe_gather_combine, *args)


def moe_shared_expert_workspace_bytes(dtype, T, I_s) -> int:
    dt = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(load().moe_shared_expert_workspace_bytes(dt, int(T), int(I_s)))


def moe_shared_expert(x, ws1, ws2, w_gate, y, workspace, accumulate=True, stream=None, layout=MOE_W_KN):
    lib = load()
    T, H = x.shape
    nk = layout == MOE_W_NK
    I_s = ws2.shape[1] if nk else ws2.shape[0]
    dev = x.device
    args = (_dt(x), int(layout), _ptr(x, "x"),
            _ptr(ws1, "ws1", x.dtype, (2 * I_s, H) if nk else (H, 2 * I_s), dev),
            _ptr(ws2, "ws2", x.dtype, (H, I_s) if nk else (I_s, H), dev),
            _ptr(w_gate, "w_gate", x.dtype, (H,), dev), T, H, I_s,
            int(bool(accumulate)), _ptr(y, "y", torch.float32, (T, H), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_shared_expert, *args)


def moe_grouped_swiglu_fc1_mx8(x_scattered, expert_offsets, w1q, w1s, act, stream=None):
    """fc1 + SwiGLU with MXFP8 weights: w1q [E, 2I, H] e4m3 codes, w1s [E, 2I/8, H] e8m0 scales (uint8)."""
    lib = load()
    R, H = x_scattered.shape
    E, I2, _ = w1q.shape
    I = I2 // 2
    dev = x_scattered.device
    u8 = torch.uint8
    args = (_ptr(x_scattered, "x_scattered", torch.bfloat16, (R, H), dev),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w1q, "w1q", u8, (E, 2 * I, H), dev), _ptr(w1s, "w1s", u8, (E, 2 * I // 8, H), dev), R, H, E, I,
            _ptr(act, "act", torch.bfloat16, (R, I), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_swiglu_fc1_mx8, *args)


def moe_grouped_fc2_mx8(act, expert_offsets, w2q, w2s, y_rows, stream=None):
    """fc2 with MXFP8 weights: w2q [E, H, I] e4m3 codes, w2s [E, H, I/8] e8m0 scales (uint8)."""
    lib = load()
    R, I = act.shape
    E, H, _ = w2q.shape
    dev = act.device
    u8 = torch.uint8
    args = (_ptr(act, "act", torch.bfloat16, (R, I), dev),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w2q, "w2q", u8, (E, H, I), dev), _ptr(w2s, "w2s", u8, (E, H, I // 8), dev), R, I, E, H,
            _ptr(y_rows, "y_rows", torch.float32, (R, H), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_fc2_mx8, *args)


def moe_shared_expert_mx8(x, ws1q, ws1s, ws2q, ws2s, w_gate, y, workspace, accumulate=True, stream=None):
    """Shared expert with MXFP8 weights: ws1q [2I_s, H] / ws1s [2I_s/8, H], ws2q [H, I_s] / ws2s [H, I_s/8]."""
    lib = load()
    T, H = x.shape
    I_s = ws2q.shape[1]
    dev = x.device
    u8 = torch.uint8
    args = (_ptr(x, "x", torch.bfloat16, (T, H), dev), _ptr(ws1q, "ws1q", u8, (2 * I_s, H), dev),
            _ptr(ws1s, "ws1s", u8, (2 * I_s // 8, H), dev), _ptr(ws2q, "ws2q", u8, (H, I_s), dev),
            _ptr(ws2s, "ws2s", u8, (H, I_s // 8), dev), _ptr(w_gate, "w_gate", torch.bfloat16, (H,), dev), T, H,
            I_s, int(bool(accumulate)), _ptr(y, "y", torch.float32, (T, H), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_shared_expert_mx8, *args)


def moe_grouped_swiglu_fc1_and_shared_mx8(x_scattered, expert_offsets, w1q, w1s, act, x, ws1q, ws1s, act_shared,
                                          stream=None):
    lib = load()
    R, H = x_scattered.shape
    E, I2, _ = w1q.shape
    I = I2 // 2
    T = x.shape[0]
    I_s = ws1q.shape[0] // 2
    dev = x.device
    u8, b16 = torch.uint8, torch.bfloat16
    args = (_ptr(x_scattered, "x_scattered", b16, (R, H), dev),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w1q, "w1q", u8, (E, 2 * I, H), dev), _ptr(w1s, "w1s", u8, (E, 2 * I // 8, H), dev), R, H, E, I,
            _ptr(act, "act", b16, (R, I), dev), _ptr(x, "x", b16, (T, H), dev),
            _ptr(ws1q, "ws1q", u8, (2 * I_s, H), dev), _ptr(ws1s, "ws1s", u8, (2 * I_s // 8, H), dev), T, I_s,
            _ptr(act_shared, "act_shared", b16, (T, I_s), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_swiglu_fc1_and_shared_mx8, *args)


def moe_grouped_fc2_and_shared_mx8(act, expert_offsets, w2q, w2s, y_rows, act_shared, ws2q, ws2s, x, w_gate, y,
                                   workspace, accumulate=False, stream=None):
    lib = load()
    R, I = act.shape
    E, H, _ = w2q.shape
    T, I_s = act_shared.shape
    dev = act.device
    u8, b16 = torch.uint8, torch.bfloat16
    args = (_ptr(act, "act", b16, (R, I), dev), _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w2q, "w2q", u8, (E, H, I), dev), _ptr(w2s, "w2s", u8, (E, H, I // 8), dev), R, I, E, H,
            _ptr(y_rows, "y_rows", torch.float32, (R, H), dev), _ptr(act_shared, "act_shared", b16, (T, I_s), dev),
            _ptr(ws2q, "ws2q", u8, (H, I_s), dev), _ptr(ws2s, "ws2s", u8, (H, I_s // 8), dev),
            _ptr(x, "x", b16, (T, H), dev), _ptr(w_gate, "w_gate", b16, (H,), dev), T, I_s, int(bool(accumulate)),
            _ptr(y, "y", torch.float32, (T, H), dev), _ptr(workspace, "workspace", torch.uint8, None, dev),
            workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_fc2_and_shared_mx8, *args)


(MOE_TILE_F32, MOE_TILE_GENERIC, MOE_TILE_128x128, MOE_TILE_256x256, MOE_TILE_128x256, MOE_TILE_32x128,
 MOE_TILE_128x512, MOE_TILE_32x64) = range(8)


def moe_grouped_gemm_tile(dtype, call, R, H, E, I, T=0, I_s=0) -> int:
    """moe_tile_config of the routed experts' launch of fc1 (call 0) or fc2 (call 1) for these sizes."""
    dt = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(load().moe_grouped_gemm_tile(dt, int(call), int(R), int(H), int(E), int(I), int(T), int(I_s)))


def moe_and_shared_launches(dtype, R, H, E, I, T, I_s) -> int:
    dt = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(load().moe_and_shared_launches(dt, int(R), int(H), int(E), int(I), int(T), int(I_s)))


def moe_grouped_swiglu_fc1_and_shared(x_scattered, expert_offsets, w1, act, x, ws1, act_shared, stream=None,
                                      layout=MOE_W_KN):
    lib = load()
    R, H = x_scattered.shape
    E, _, I = _fc1_sizes(w1, layout)
    nk = layout == MOE_W_NK
    T = x.shape[0]
    I_s = (ws1.shape[0] if nk else ws1.shape[1]) // 2
    dev = x.device
    dt = x.dtype
    args = (_dt(x), int(layout), _ptr(x_scattered, "x_scattered", dt, (R, H), dev),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w1, "w1", dt, (E, 2 * I, H) if nk else (E, H, 2 * I), dev), R, H, E, I,
            _ptr(act, "act", dt, (R, I), dev), _ptr(x, "x", dt, (T, H), dev),
            _ptr(ws1, "ws1", dt, (2 * I_s, H) if nk else (H, 2 * I_s), dev), T, I_s,
            _ptr(act_shared, "act_shared", dt, (T, I_s), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_swiglu_fc1_and_shared, *args)


def moe_grouped_swiglu_fc1_and_shared_gather(x, row_token, expert_offsets, w1, act, ws1, act_shared, stream=None,
                                             layout=MOE_W_KN):
    """moe_grouped_swiglu_fc1_and_shared reading routed row r as x[row_token[r]] (no x_scattered)."""
    lib = load()
    T, H = x.shape
    R = row_token.shape[0]
    E, _, I = _fc1_sizes(w1, layout)
    nk = layout == MOE_W_NK
    I_s = (ws1.shape[0] if nk else ws1.shape[1]) // 2
    dev = x.device
    dt = x.dtype
    args = (_dt(x), int(layout), _ptr(x, "x", dt, (T, H), dev), _ptr(row_token, "row_token", torch.int32, (R,), dev),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w1, "w1", dt, (E, 2 * I, H) if nk else (E, H, 2 * I), dev), R, H, E, I,
            _ptr(act, "act", dt, (R, I), dev),
            _ptr(ws1, "ws1", dt, (2 * I_s, H) if nk else (H, 2 * I_s), dev), T, I_s,
            _ptr(act_shared, "act_shared", dt, (T, I_s), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_swiglu_fc1_and_shared_gather, *args)


def moe_grouped_fc2_and_shared(act, expert_offsets, w2, y_rows, act_shared, ws2, x, w_gate, y, workspace,
                               accumulate=False, stream=None, layout=MOE_W_KN):
    lib = load()
    R, I = act.shape
    nk = layout == MOE_W_NK
    E = w2.shape[0]
    H = w2.shape[1] if nk else w2.shape[2]
    T, I_s = act_shared.shape
    dev = act.device
    dt = act.dtype
    args = (_dt(act), int(layout), _ptr(act, "act"),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w2, "w2", dt, (E, H, I) if nk else (E, I, H), dev), R, I, E, H,
            _ptr(y_rows, "y_rows", torch.float32, (R, H), dev),
            _ptr(act_shared, "act_shared", dt, (T, I_s), dev),
            _ptr(ws2, "ws2", dt, (H, I_s) if nk else (I_s, H), dev),
            _ptr(x, "x", dt, (T, H), dev), _ptr(w_gate, "w_gate", dt, (H,), dev), T, I_s, int(bool(accumulate)),
            _ptr(y, "y", torch.float32, (T, H), dev), _ptr(workspace, "workspace", torch.uint8, None, dev),
            workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_fc2_and_shared, *args)


class MoELayerBuffers:
    """Device buffers for one layer forward of T tokens (allocated once, reused)."""

    def __init__(self, T, H, E, top_k, I, I_s, dtype, device):
        R = T * top_k
        i32, f32 = torch.int32, torch.float32
        self.T, self.H, self.E, self.top_k, self.I, self.I_s = T, H, E, top_k, I, I_s
        self.logits = torch.empty((T, E), dtype=f32, device=device)
        self.topk_ids = torch.empty((T, top_k), dtype=i32, device=device)
        self.topk_weights = torch.empty((T, top_k), dtype=f32, device=device)
        self.scatter_index = torch.empty((T, top_k), dtype=i32, device=device)
        self.row_token = torch.empty((R,), dtype=i32, device=device)
        self.expert_offsets = torch.empty((E + 1,), dtype=i32, device=device)
        self.status_words = torch.zeros((2,), dtype=i32, device=device)
        self.x_scattered = torch.empty((R, H), dtype=dtype, device=device)
        self.act = torch.empty((R, I), dtype=dtype, device=device)
        self.y_rows = torch.empty((R, H), dtype=f32, device=device)
        self.y = torch.empty((T, H), dtype=f32, device=device)
        rb = moe_route_workspace_bytes(dtype, T, H, E)
        self.route_ws = torch.empty((max(rb, 1),), dtype=torch.uint8, device=device)
        self.scatter_ws = torch.empty((moe_build_scatter_workspace_bytes(T, top_k, E),), dtype=torch.uint8,
                                      device=device)
        self.route_scatter_ws = torch.empty((moe_route_and_scatter_workspace_bytes(dtype, T, H, E, top_k),),
                                            dtype=torch.uint8, device=device)
        self.shared_ws = (torch.empty((moe_shared_expert_workspace_bytes(dtype, T, I_s),), dtype=torch.uint8,
                                      device=device) if I_s > 0 else None)
        self.act_shared = torch.empty((T, I_s), dtype=dtype, device=device) if I_s > 0 else None


def moe_layer_forward(x, w_router, logit_bias, W1, W2, top_k, shared=None, bufs=None, routes=None,
                      stream=None, fused_shared=False, fused_route=False, side_stream=None, layout=MOE_W_KN,
                      gather=False):
    """The six calls in order.  ``routes`` = (topk_ids int32, topk_weights fp32)
    device tensors skips moe_route.  ``shared`` = (ws1, ws2, w_gate or None).
    With ``fused_shared`` and a shared expert, the routed experts and the shared
    expert run together through moe_grouped_swiglu_fc1_and_shared and
    moe_grouped_fc2_and_shared, and the combine adds the routed outputs onto the
    shared ones.  With ``fused_route`` (and no fed-in routes), routing and the
    scatter build run through moe_route_and_scatter.  With ``side_stream`` (a
    torch.cuda.Stream; not with ``fused_shared``) and a shared expert, the shared
    expert runs there first (y = shared(x)), concurrently with routing and the
    routed experts, and the combine waits for it and adds onto y.  ``layout``
    (MOE_W_KN or MOE_W_NK) is the storage of W1, W2 and the shared weights.  With
    ``gather`` the scatter build copies no rows (x_scattered NULL) and fc1 reads
    the routed rows from x through row_token (the *_gather calls)."""
    T, H = x.shape
    E, _, I = _fc1_sizes(W1, layout)
    I_s = (shared[1].shape[1] if layout == MOE_W_NK else shared[1].shape[0]) if shared is not None else 0
    if bufs is None:
        bufs = MoELayerBuffers(T, H, E, top_k, I, I_s, x.dtype, x.device)
    if routes is None and fused_route:
        moe_route_and_scatter(x, w_router, logit_bias, top_k, bufs.topk_ids, bufs.topk_weights, bufs.logits,
                              bufs.scatter_index, bufs.row_token, bufs.expert_offsets, bufs.status_words,
                              None if gather else bufs.x_scattered, bufs.route_scatter_ws, stream)
        w = bufs.topk_weights
    else:
        if routes is None:
            moe_route(x, w_router, logit_bias, top_k, bufs.topk_ids, bufs.topk_weights, bufs.logits, bufs.route_ws,
                      stream)
            ids, w = bufs.topk_ids, bufs.topk_weights
        else:
            ids, w = routes
        moe_build_scatter(x, ids, E, bufs.scatter_index, bufs.row_token, bufs.expert_offsets, bufs.status_words,
                          None if gather else bufs.x_scattered, bufs.scatter_ws, stream)
    if side_stream is not None and shared is not None and not fused_shared:
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            raise ValueError("side_stream needs stream to be None or a torch.cuda.Stream")
        main = torch.cuda.current_stream(x.device) if stream is None else stream
        side_stream.wait_stream(main)
        ws1, ws2, wg = shared
        moe_shared_expert(x, ws1, ws2, wg, bufs.y, bufs.shared_ws, False, side_stream, layout=layout)
    if fused_shared and shared is not None:
        ws1, ws2, wg = shared
        if gather:
            moe_grouped_swiglu_fc1_and_shared_gather(x, bufs.row_token, bufs.expert_offsets, W1, bufs.act, ws1,
                                                     bufs.act_shared, stream, layout=layout)
        else:
            moe_grouped_swiglu_fc1_and_shared(bufs.x_scattered, bufs.expert_offsets, W1, bufs.act, x, ws1,
                                              bufs.act_shared, stream, layout=layout)
        moe_grouped_fc2_and_shared(bufs.act, bufs.expert_offsets, W2, bufs.y_rows, bufs.act_shared, ws2, x, wg,
                                   bufs.y, bufs.shared_ws, False, stream, layout=layout)
        moe_gather_combine(bufs.y_rows, bufs.scatter_index, w, bufs.y, True, stream)
        return bufs
    if gather:
        moe_grouped_swiglu_fc1_gather(x, bufs.row_token, bufs.expert_offsets, W1, bufs.act, stream, layout=layout)
    else:
        moe_grouped_swiglu_fc1(bufs.x_scattered, bufs.expert_offsets, W1, bufs.act, stream, layout=layout)
    moe_grouped_fc2(bufs.act, bufs.expert_offsets, W2, bufs.y_rows, stream, layout=layout)
    if side_stream is not None and shared is not None:
        main.wait_stream(side_stream)
        moe_gather_combine(bufs.y_rows, bufs.scatter_index, w, bufs.y, True, stream)
        return bufs
    moe_gather_combine(bufs.y_rows, bufs.scatter_index, w, bufs.y, False, stream)
    if shared is not None:
        ws1, ws2, wg = shared
        moe_shared_expert(x, ws1, ws2, wg, bufs.y, bufs.shared_ws, True, stream, layout=layout)
    return bufs


# ------------------------------------------------------------------------------------------
# Backward of the routed experts
# ------------------------------------------------------------------------------------------
def _w1_shape(E, H, I, layout):
    return (E, 2 * I, H) if layout == MOE_W_NK else (E, H, 2 * I)


def _w2_shape(E, H, I, layout):
    return (E, H, I) if layout == MOE_W_NK else (E, I, H)


def moe_grouped_swiglu_fc1_save(x_scattered, expert_offsets, w1, act, h_pre, stream=None, layout=MOE_W_KN):
    lib = load()
    R, H = x_scattered.shape
    E, _, I = _fc1_sizes(w1, layout)
    dev = x_scattered.device
    dt = x_scattered.dtype
    args = (_dt(x_scattered), int(layout), _ptr(x_scattered, "x_scattered"),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w1, "w1", dt, _w1_shape(E, H, I, layout), dev), R, H, E, I,
            _ptr(act, "act", dt, (R, I), dev), _ptr(h_pre, "h_pre", dt, (R, 2 * I), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_swiglu_fc1_save, *args)


def moe_scatter_grad(dy, y_rows, topk_weights, scatter_index, d_rows, d_topk_weights, stream=None):
    lib = load()
    T, H = dy.shape
    k = scatter_index.shape[1]
    R = y_rows.shape[0]
    dev = dy.device
    args = (_dt(d_rows), _ptr(dy, "dy", torch.float32, (T, H), dev),
            _ptr(y_rows, "y_rows", torch.float32, (R, H), dev),
            _ptr(topk_weights, "topk_weights", torch.float32, (T, k), dev),
            _ptr(scatter_index, "scatter_index", torch.int32, (T, k), dev), T, H, k, R,
            _ptr(d_rows, "d_rows", None, (R, H), dev),
            _ptr(d_topk_weights, "d_topk_weights", torch.float32, (T, k), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_scatter_grad, *args)


def moe_grouped_fc2_backward(d_rows, act, h_pre, expert_offsets, w2, d_h, d_w2, stream=None, layout=MOE_W_KN):
    lib = load()
    R, I = act.shape
    H = d_rows.shape[1]
    E = w2.shape[0]
    dev = act.device
    dt = act.dtype
    args = (_dt(act), int(layout), _ptr(d_rows, "d_rows", dt, (R, H), dev), _ptr(act, "act"),
            _ptr(h_pre, "h_pre", dt, (R, 2 * I), dev),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w2, "w2", dt, _w2_shape(E, H, I, layout), dev), R, I, E, H,
            _ptr(d_h, "d_h", dt, (R, 2 * I), dev), _ptr(d_w2, "d_w2", dt, _w2_shape(E, H, I, layout), dev),
            _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_fc2_backward, *args)


def moe_grouped_fc1_backward_workspace_bytes(R, H) -> int:
    return int(load().moe_grouped_fc1_backward_workspace_bytes(int(R), int(H)))


def moe_grouped_fc1_backward(d_h, x_scattered, expert_offsets, w1, scatter_index, d_x, d_w1, workspace,
                             accumulate=False, stream=None, layout=MOE_W_KN):
    lib = load()
    R, H = x_scattered.shape
    E, _, I = _fc1_sizes(w1, layout)
    T, k = scatter_index.shape
    dev = x_scattered.device
    dt = x_scattered.dtype
    args = (_dt(x_scattered), int(layout), _ptr(d_h, "d_h", dt, (R, 2 * I), dev), _ptr(x_scattered, "x_scattered"),
            _ptr(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev),
            _ptr(w1, "w1", dt, _w1_shape(E, H, I, layout), dev), R, H, E, I,
            _ptr(scatter_index, "scatter_index", torch.int32, (T, k), dev), T, k, int(bool(accumulate)),
            _ptr(d_x, "d_x", torch.float32, (T, H), dev), _ptr(d_w1, "d_w1", dt, _w1_shape(E, H, I, layout), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_grouped_fc1_backward, *args)


class MoEBackwardBuffers:
    """Device buffers of the routed experts' training forward and backward for T tokens."""

    def __init__(self, T, H, E, top_k, I, dtype, device, layout=MOE_W_KN):
        R = T * top_k
        f32 = torch.float32
        self.h_pre = torch.empty((R, 2 * I), dtype=dtype, device=device)
        self.d_rows = torch.empty((R, H), dtype=dtype, device=device)
        self.d_topk_weights = torch.empty((T, top_k), dtype=f32, device=device)
        self.d_h = torch.empty((R, 2 * I), dtype=dtype, device=device)
        self.d_x = torch.empty((T, H), dtype=f32, device=device)
        self.d_w1 = torch.empty(_w1_shape(E, H, I, layout), dtype=dtype, device=device)
        self.d_w2 = torch.empty(_w2_shape(E, H, I, layout), dtype=dtype, device=device)
        self.ws = torch.empty((moe_grouped_fc1_backward_workspace_bytes(R, H),), dtype=torch.uint8, device=device)


def moe_routed_train_forward(x, W1, W2, routes, bufs, bwd, stream=None, layout=MOE_W_KN):
    """Routed part of the layer for fed-in routes (ids, weights), keeping what
    the backward needs: scatter -> fc1 (saving h_pre) -> fc2 -> combine into bufs.y."""
    E = W1.shape[0]
    ids, w = routes
    moe_build_scatter(x, ids, E, bufs.scatter_index, bufs.row_token, bufs.expert_offsets, bufs.status_words,
                      bufs.x_scattered, bufs.scatter_ws, stream)
    moe_grouped_swiglu_fc1_save(bufs.x_scattered, bufs.expert_offsets, W1, bufs.act, bwd.h_pre, stream, layout=layout)
    moe_grouped_fc2(bufs.act, bufs.expert_offsets, W2, bufs.y_rows, stream, layout=layout)
    moe_gather_combine(bufs.y_rows, bufs.scatter_index, w, bufs.y, False, stream)


def moe_routed_backward(dy, W1, W2, topk_weights, bufs, bwd, stream=None, layout=MOE_W_KN):
    """The three backward calls after moe_routed_train_forward: gradients into
    bwd.d_x, bwd.d_w1, bwd.d_w2 and bwd.d_topk_weights."""
    moe_scatter_grad(dy, bufs.y_rows, topk_weights, bufs.scatter_index, bwd.d_rows, bwd.d_topk_weights, stream)
    moe_grouped_fc2_backward(bwd.d_rows, bufs.act, bwd.h_pre, bufs.expert_offsets, W2, bwd.d_h, bwd.d_w2, stream,
                             layout=layout)
    moe_grouped_fc1_backward(bwd.d_h, bufs.x_scattered, bufs.expert_offsets, W1, bufs.scatter_index, bwd.d_x,
                             bwd.d_w1, bwd.ws, False, stream, layout=layout)


# ------------------------------------------------------------------------------------------
# Training of the shared expert, backward of the router, gradient norm and clipping
# ------------------------------------------------------------------------------------------
def _ws1_shape(H, I_s, layout):
    return (2 * I_s, H) if layout == MOE_W_NK else (H, 2 * I_s)


def _ws2_shape(H, I_s, layout):
    return (H, I_s) if layout == MOE_W_NK else (I_s, H)


def moe_shared_train_workspace_bytes(dtype, T, H, I_s) -> int:
    """Workspace bytes that any of the four moe_shared_* training calls needs."""
    dt = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(load().moe_shared_train_workspace_bytes(dt, int(T), int(H), int(I_s)))


(MOE_DENSE_F32, MOE_DENSE_256x256, MOE_DENSE_128x128, MOE_DENSE_64x128, MOE_DENSE_64x128_K2,
 MOE_DENSE_64x128_128x128, MOE_DENSE_128x128_K2, MOE_DENSE_64x64_K4, MOE_DENSE_64x64_K4_128x128_K2) = range(9)


def moe_shared_train_tiles(dtype, call, T, H, I_s, layout=MOE_W_KN):
    """(moe_dense_tiles, splits of the input side, splits of the weight gradient) of a training call of the shared
    expert (0 fc1_save, 1 fc2_save, 2 fc2_backward, 3 fc1_backward)."""
    dt = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    splits = (_c_int * 2)()
    r = load().moe_shared_train_tiles(dt, int(call), int(layout), int(T), int(H), int(I_s), splits)
    return int(r), splits[0], splits[1]


def moe_shared_fc1_save(x, ws1, act, h_pre, workspace, stream=None, layout=MOE_W_KN):
    """Shared fc1 + SwiGLU keeping the pre-activation: act [T, I_s], h_pre [T, 2 I_s] = [g | u]."""
    lib = load()
    T, H = x.shape
    I_s = act.shape[1]
    dev, dt = x.device, x.dtype
    args = (_dt(x), int(layout), _ptr(x, "x"), _ptr(ws1, "ws1", dt, _ws1_shape(H, I_s, layout), dev), T, H, I_s,
            _ptr(act, "act", dt, (T, I_s), dev), _ptr(h_pre, "h_pre", dt, (T, 2 * I_s), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_shared_fc1_save, *args)


def moe_shared_fc2_save(act, ws2, x, w_gate, y, y_shared, gate, workspace, accumulate=False, stream=None,
                        layout=MOE_W_KN):
    """Shared fc2 and gate onto y [T, H] (fp32).  Gated (w_gate given): also y_shared [T, H] and gate [T] (fp32);
    ungated: y_shared and gate are None and x is not used."""
    lib = load()
    T, I_s = act.shape
    H = y.shape[1]
    dev, dt, f32 = act.device, act.dtype, torch.float32
    args = (_dt(act), int(layout), _ptr(act, "act"), _ptr(ws2, "ws2", dt, _ws2_shape(H, I_s, layout), dev),
            _ptr(x, "x", dt, (T, H), dev), _ptr(w_gate, "w_gate", dt, (H,), dev), T, H, I_s, int(bool(accumulate)),
            _ptr(y, "y", f32, (T, H), dev), _ptr(y_shared, "y_shared", f32, (T, H), dev),
            _ptr(gate, "gate", f32, (T,), dev), _ptr(workspace, "workspace", torch.uint8, None, dev),
            workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_shared_fc2_save, *args)


def moe_shared_fc2_backward(dy, act, h_pre, ws2, y_shared, gate, d_h, d_ws2, d_gate_logit, workspace, stream=None,
                            layout=MOE_W_KN):
    """Gradients through the gate, fc2 and SwiGLU: d_h [T, 2 I_s], d_ws2, and with a gate d_gate_logit [T] (fp32).
    Ungated: y_shared, gate and d_gate_logit are None."""
    lib = load()
    T, I_s = act.shape
    H = dy.shape[1]
    dev, dt, f32 = act.device, act.dtype, torch.float32
    args = (_dt(act), int(layout), _ptr(dy, "dy", f32, (T, H), dev), _ptr(act, "act"),
            _ptr(h_pre, "h_pre", dt, (T, 2 * I_s), dev), _ptr(ws2, "ws2", dt, _ws2_shape(H, I_s, layout), dev),
            _ptr(y_shared, "y_shared", f32, (T, H), dev), _ptr(gate, "gate", f32, (T,), dev), T, H, I_s,
            _ptr(d_h, "d_h", dt, (T, 2 * I_s), dev), _ptr(d_ws2, "d_ws2", dt, _ws2_shape(H, I_s, layout), dev),
            _ptr(d_gate_logit, "d_gate_logit", f32, (T,), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_shared_fc2_backward, *args)


def moe_shared_fc1_backward(d_h, x, ws1, d_gate_logit, w_gate, d_x, d_ws1, d_w_gate, workspace, accumulate=False,
                            stream=None, layout=MOE_W_KN):
    """Gradients through fc1 and the gate's dot product: d_x [T, H] (fp32, optionally added to), d_ws1, d_w_gate [H].
    Ungated: d_gate_logit, w_gate and d_w_gate are None."""
    lib = load()
    T, H = x.shape
    I_s = d_h.shape[1] // 2
    dev, dt, f32 = x.device, x.dtype, torch.float32
    args = (_dt(x), int(layout), _ptr(d_h, "d_h", dt, (T, 2 * I_s), dev), _ptr(x, "x"),
            _ptr(ws1, "ws1", dt, _ws1_shape(H, I_s, layout), dev),
            _ptr(d_gate_logit, "d_gate_logit", f32, (T,), dev), _ptr(w_gate, "w_gate", dt, (H,), dev), T, H, I_s,
            int(bool(accumulate)), _ptr(d_x, "d_x", f32, (T, H), dev),
            _ptr(d_ws1, "d_ws1", dt, _ws1_shape(H, I_s, layout), dev), _ptr(d_w_gate, "d_w_gate", dt, (H,), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_shared_fc1_backward, *args)


def moe_route_backward_workspace_bytes(dtype, T, H, E, top_k) -> int:
    dt = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(load().moe_route_backward_workspace_bytes(dt, int(T), int(H), int(E), int(top_k)))


def moe_route_backward(x, w_router, topk_ids, topk_weights, d_topk_weights, d_x, d_w_router, d_logit_bias, workspace,
                       accumulate=False, stream=None):
    """Gradients of the router: d_x [T, H] (fp32, optionally added to), d_w_router [H, E] and d_logit_bias [E] (fp32,
    or None) from the route weights' gradient d_topk_weights [T, top_k]."""
    lib = load()
    T, H = x.shape
    E = w_router.shape[1]
    k = topk_ids.shape[1]
    dev, dt, f32 = x.device, x.dtype, torch.float32
    args = (_dt(x), _ptr(x, "x"), _ptr(w_router, "w_router", dt, (H, E), dev),
            _ptr(topk_ids, "topk_ids", torch.int32, (T, k), dev),
            _ptr(topk_weights, "topk_weights", f32, (T, k), dev),
            _ptr(d_topk_weights, "d_topk_weights", f32, (T, k), dev), T, H, E, k, int(bool(accumulate)),
            _ptr(d_x, "d_x", f32, (T, H), dev), _ptr(d_w_router, "d_w_router", dt, (H, E), dev),
            _ptr(d_logit_bias, "d_logit_bias", f32, (E,), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_route_backward, *args)


class MoEGradList:
    """A list of gradient tensors as moe_grad_norm and moe_grad_clip take it: checked once, its pointers marshalled
    once.  ``grads`` are contiguous float32 or bfloat16 tensors of one device (any shape); ``outs`` (default: the
    gradients themselves, scaled in place) are what moe_grad_clip writes, of the same types and sizes.  The list
    refers to the tensors' memory and keeps them alive; make a new one when a tensor is replaced."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        n = len(self.grads)
        if n < 1 or len(self.outs) != n:
            raise ValueError(f"a gradient list needs at least one tensor and as many outputs (got {n} and "
                             f"{len(self.outs)})")
        dev = self.grads[0].device
        self.device = dev
        self._in = (_vp * n)(*[_ptr(g, f"grads[{i}]", None, None, dev) for i, g in enumerate(self.grads)])
        self._out = (_vp * n)(*[_ptr(o, f"outs[{i}]", g.dtype, None, dev)
                                for i, (g, o) in enumerate(zip(self.grads, self.outs))])
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            if g.numel() != o.numel():
                raise ValueError(f"outs[{i}] must have {g.numel()} elements (got {o.numel()})")
        self._numel = (ctypes.c_int64 * n)(*[g.numel() for g in self.grads])
        self._dts = (_c_int * n)(*[_dt(g) for g in self.grads])
        self.n = n


def moe_grad_norm_workspace_bytes(n) -> int:
    return int(load().moe_grad_norm_workspace_bytes(int(n)))


def moe_grad_norm(grads, norm, workspace, sum_sq=None, stream=None):
    """2-norm of all gradients of a MoEGradList taken together into norm [1] (fp32), and the sum of squares into
    sum_sq [1] (fp64) if given."""
    lib = load()
    dev = grads.device
    args = (grads.n, grads._in, grads._numel, grads._dts, _ptr(norm, "norm", torch.float32, (1,), dev),
            _ptr(sum_sq, "sum_sq", torch.float64, (1,), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_grad_norm, *args)


def moe_grad_clip(grads, norm, max_norm, coef=None, stream=None):
    """Scales the gradients of a MoEGradList by min(1, max_norm / (norm + 1e-6)) into its outputs; norm [1] (fp32,
    device) as moe_grad_norm left it, coef [1] (fp32) receives the factor if given."""
    lib = load()
    dev = grads.device
    args = (grads.n, grads._in, grads._out, grads._numel, grads._dts, _ptr(norm, "norm", torch.float32, (1,), dev),
            float(max_norm), _ptr(coef, "coef", torch.float32, (1,), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_grad_clip, *args)


class MoETrainBuffers(MoEBackwardBuffers):
    """Device buffers of a whole layer's training step for T tokens: those of the routed experts' backward, and
    what the shared expert (I_s > 0, gated or not) and the router need."""

    def __init__(self, T, H, E, top_k, I, I_s, gated, has_bias, dtype, device, layout=MOE_W_KN):
        super().__init__(T, H, E, top_k, I, dtype, device, layout)
        f32 = torch.float32
        new = lambda shape, dt=dtype: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        self.d_w_router = new((H, E))
        self.d_logit_bias = new((E,), f32) if has_bias else None
        with torch.cuda.device(device):   # the workspace goes by the device's compute units
            self.route_ws = new((moe_route_backward_workspace_bytes(dtype, T, H, E, top_k),), torch.uint8)
        self.I_s, self.gated = I_s, gated
        self.d_ws1 = self.d_ws2 = self.d_w_gate = None
        self.y_shared = self.gate = self.d_gate_logit = None
        if I_s > 0:
            self.act_shared, self.h_shared, self.d_h_shared = new((T, I_s)), new((T, 2 * I_s)), new((T, 2 * I_s))
            self.d_ws1, self.d_ws2 = new(_ws1_shape(H, I_s, layout)), new(_ws2_shape(H, I_s, layout))
            self.shared_ws = new((moe_shared_train_workspace_bytes(dtype, T, H, I_s),), torch.uint8)
            if gated:
                self.y_shared, self.gate, self.d_gate_logit = new((T, H), f32), new((T,), f32), new((T,), f32)
                self.d_w_gate = new((H,))
        self.norm, self.coef = new((1,), f32), new((1,), f32)
        self._grads = None
        self.norm_ws = new((moe_grad_norm_workspace_bytes(self.grads.n),), torch.uint8)

    def grad_tensors(self):
        """What ``grads`` lists: the gradients of the layer's parameters as they are now, or those of a list set there."""
        if self._grads is not None:
            return self._grads.grads
        return [g for g in (self.d_w1, self.d_w2, self.d_w_router, self.d_logit_bias, self.d_ws1, self.d_ws2,
                            self.d_w_gate) if g is not None]

    @property
    def grads(self):
        """The gradients that moe_layer_backward clips, as one MoEGradList.  It is made for every call (9 us): a list
        that was kept would go on scaling a tensor that has been replaced here.  A list that is set is taken as it is."""
        return MoEGradList(self.grad_tensors()) if self._grads is None else self._grads

    @grads.setter
    def grads(self, grads):
        self._grads = grads


def _need_layer(train, shared):
    have = "no shared expert" if train.I_s == 0 else f"a shared expert {'with' if train.gated else 'without'} a gate"
    want = "no shared expert" if shared is None else (
        f"a shared expert {'without' if shared[2] is None else 'with'} a gate")
    if have != want:
        raise ValueError(f"the training buffers were made for a layer with {have} (called with {want})")


def moe_layer_train_forward(x, w_router, logit_bias, W1, W2, top_k, shared, bufs, train, stream=None,
                            layout=MOE_W_KN):
    """Training forward of the whole layer into bufs.y: routing, the routed experts and the shared expert
    (``shared`` = (ws1, ws2, w_gate or None), or None), keeping in ``bufs`` (MoELayerBuffers) and ``train``
    (MoETrainBuffers) what moe_layer_backward needs."""
    _need_layer(train, shared)
    if (logit_bias is None) != (train.d_logit_bias is None):
        raise ValueError("the training buffers were made for a router "
                         f"{'with' if logit_bias is None else 'without'} a logit bias")
    moe_route(x, w_router, logit_bias, top_k, bufs.topk_ids, bufs.topk_weights, bufs.logits, bufs.route_ws, stream)
    moe_routed_train_forward(x, W1, W2, (bufs.topk_ids, bufs.topk_weights), bufs, train, stream, layout)
    if shared is not None:
        ws1, ws2, wg = shared
        moe_shared_fc1_save(x, ws1, train.act_shared, train.h_shared, train.shared_ws, stream, layout=layout)
        moe_shared_fc2_save(train.act_shared, ws2, x, wg, bufs.y, train.y_shared, train.gate, train.shared_ws, True,
                            stream, layout=layout)
    return bufs


class MoERouteLosses(NamedTuple):
    """The router's auxiliary losses in a backward pass: ``block`` (MoEBlockBuffers) with what moe_balance_loss left,
    and its arguments."""

    block: object
    token_mask: object = None
    balance_coef: float = 0.01
    z_coef: float = 0.0


def moe_layer_backward(dy, x, w_router, W1, W2, shared, bufs, train, max_norm=None, stream=None, layout=MOE_W_KN,
                       losses=None):
    """Backward of moe_layer_train_forward from dy [T, H] (fp32): every parameter's gradient and d_x into ``train``
    (d_w1, d_w2, d_w_router, d_logit_bias, d_ws1, d_ws2, d_w_gate, d_x).  With ``max_norm`` the parameters'
    gradients are then scaled in place to at most that norm together (train.norm, train.coef).  With ``losses``
    (MoERouteLosses) the router's gradients include those of its auxiliary losses."""
    _need_layer(train, shared)
    moe_routed_backward(dy, W1, W2, bufs.topk_weights, bufs, train, stream, layout)
    if losses is None:
        moe_route_backward(x, w_router, bufs.topk_ids, bufs.topk_weights, train.d_topk_weights, train.d_x,
                           train.d_w_router, train.d_logit_bias, train.route_ws, True, stream)
    else:
        b = losses.block
        moe_route_balance_backward(x, w_router, bufs.logits, b.lse, bufs.topk_ids, bufs.topk_weights,
                                   train.d_topk_weights, losses.token_mask, b.counts, b.tokens, train.d_x,
                                   train.d_w_router, train.d_logit_bias, b.route_ws, losses.balance_coef,
                                   losses.z_coef, True, stream)
    if shared is not None:
        ws1, ws2, wg = shared
        moe_shared_fc2_backward(dy, train.act_shared, train.h_shared, ws2, train.y_shared, train.gate,
                                train.d_h_shared, train.d_ws2, train.d_gate_logit, train.shared_ws, stream,
                                layout=layout)
        moe_shared_fc1_backward(train.d_h_shared, x, ws1, train.d_gate_logit, wg, train.d_x, train.d_ws1,
                                train.d_w_gate, train.shared_ws, True, stream, layout=layout)
    if max_norm is not None:
        grads = train.grads
        moe_grad_norm(grads, train.norm, train.norm_ws, stream=stream)
        moe_grad_clip(grads, train.norm, max_norm, train.coef, stream=stream)
    return train


# ------------------------------------------------------------------------------------------
# Around the layer: auxiliary losses of the router, norms and residual, orthogonalised update
# ------------------------------------------------------------------------------------------
def _dtype_id(dtype) -> int:
    return MOE_BF16 if dtype == torch.bfloat16 else MOE_F32


def _mask_ptr(mask, T, dev):
    """A token mask: torch.bool or torch.uint8, one byte per token."""
    if mask is not None and mask.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"token_mask must be torch.bool or torch.uint8 (got {mask.dtype})")
    return _ptr(mask, "token_mask", None, (T,), dev)


def moe_balance_loss_workspace_bytes(T, E) -> int:
    return int(load().moe_balance_loss_workspace_bytes(int(T), int(E)))


def moe_balance_loss(logits, topk_ids, token_mask, losses, counts, tokens, prob_sums, lse, workspace,
                     balance_coef=0.01, z_coef=0.0, stream=None):
    """Balance and z loss of a batch's routes into losses [2] (fp32), with counts [E] (int32), tokens [1] (int32, the
    valid ones), prob_sums [E] and lse [T] (fp32).  ``token_mask`` [T] (bool or uint8) or None."""
    lib = load()
    T, E = logits.shape
    k = topk_ids.shape[1]
    dev, f32, i32 = logits.device, torch.float32, torch.int32
    args = (_ptr(logits, "logits", f32), _ptr(topk_ids, "topk_ids", i32, (T, k), dev), _mask_ptr(token_mask, T, dev),
            T, E, k, float(balance_coef), float(z_coef), _ptr(losses, "losses", f32, (2,), dev),
            _ptr(counts, "counts", i32, (E,), dev), _ptr(tokens, "tokens", i32, (1,), dev),
            _ptr(prob_sums, "prob_sums", f32, (E,), dev), _ptr(lse, "lse", f32, (T,), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_balance_loss, *args)


def moe_route_balance_backward_workspace_bytes(dtype, T, H, E, top_k) -> int:
    """``top_k`` takes no space; it is here so that both router backward calls are asked alike."""
    return int(load().moe_route_balance_backward_workspace_bytes(_dtype_id(dtype), int(T), int(H), int(E)))


def moe_route_balance_backward(x, w_router, logits, lse, topk_ids, topk_weights, d_topk_weights, token_mask, counts,
                               tokens, d_x, d_w_router, d_logit_bias, workspace, balance_coef=0.01, z_coef=0.0,
                               accumulate=False, stream=None, top_k=None):
    """moe_route_backward with the gradients of moe_balance_loss's losses: d_x [T, H] (fp32, optionally added to),
    d_w_router [H, E] and d_logit_bias [E] (fp32, or None).  Without route weights (topk_weights and d_topk_weights
    None) the losses' gradients alone; topk_ids may be None too then, with the slots per token in ``top_k``."""
    lib = load()
    T, H = x.shape
    E = w_router.shape[1]
    k = top_k if topk_ids is None else topk_ids.shape[1]
    if k is None or (top_k is not None and int(top_k) != k):
        raise ValueError("top_k must be given without topk_ids" if k is None else
                         f"top_k is {top_k}, topk_ids has {k} slots per token")
    k = int(k)
    dev, dt, f32, i32 = x.device, x.dtype, torch.float32, torch.int32
    args = (_dt(x), _ptr(x, "x"), _ptr(w_router, "w_router", dt, (H, E), dev),
            _ptr(logits, "logits", f32, (T, E), dev), _ptr(lse, "lse", f32, (T,), dev),
            _ptr(topk_ids, "topk_ids", i32, (T, k), dev), _ptr(topk_weights, "topk_weights", f32, (T, k), dev),
            _ptr(d_topk_weights, "d_topk_weights", f32, (T, k), dev), _mask_ptr(token_mask, T, dev),
            _ptr(counts, "counts", i32, (E,), dev), _ptr(tokens, "tokens", i32, (1,), dev), T, H, E, k,
            float(balance_coef), float(z_coef), int(bool(accumulate)), _ptr(d_x, "d_x", f32, (T, H), dev),
            _ptr(d_w_router, "d_w_router", dt, (H, E), dev), _ptr(d_logit_bias, "d_logit_bias", f32, (E,), dev),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_route_balance_backward, *args)


def _norm_dtype(x, *weights):
    """Element type of a norm call's x and weights (that of the stream if there are none)."""
    given = [t for t in (x, *weights) if t is not None]
    return given[0] if given else None


def moe_norm_residual(h, y, w_post, gate, w_pre, h_out, x, rstd_post=None, rstd_pre=None, eps=1e-6,
                      weight_offset=0.0, residual_scale=1.0, branch_scale=1.0, stream=None):
    """h_out = residual_scale h + branch_scale gate norm(y) and x = norm(h_out) in one pass (y None: x = norm(h)).  h
    and h_out [T, H] in the stream's type, y [T, H] fp32, x [T, H] and the weights [H] of one type."""
    lib = load()
    T, H = h.shape
    dev, f32 = h.device, torch.float32
    ref = _norm_dtype(x, w_post, gate, w_pre)
    dt = h.dtype if ref is None else ref.dtype
    w = lambda t, name: _ptr(t, name, dt, (H,), dev)   # noqa: E731
    args = (_dt(h if ref is None else ref), _dt(h), _ptr(h, "h"), _ptr(y, "y", f32, (T, H), dev),
            w(w_post, "w_post"), w(gate, "gate"), w(w_pre, "w_pre"), T, H, float(eps), float(weight_offset),
            float(residual_scale), float(branch_scale), _ptr(h_out, "h_out", h.dtype, (T, H), dev),
            _ptr(x, "x", dt, (T, H), dev), _ptr(rstd_post, "rstd_post", f32, (T,), dev),
            _ptr(rstd_pre, "rstd_pre", f32, (T,), dev), _stream(stream, dev))
    _call_on(dev, lib.moe_norm_residual, *args)


def moe_norm_residual_backward_workspace_bytes(T, H) -> int:
    return int(load().moe_norm_residual_backward_workspace_bytes(int(T), int(H)))


def moe_norm_residual_backward(d_h_out, d_x, h_out, rstd_pre, w_pre, y, rstd_post, w_post, gate, d_h, d_y, d_w_pre,
                               d_w_post, d_gate, workspace, weight_offset=0.0, residual_scale=1.0, branch_scale=1.0,
                               stream=None):
    """Gradients of moe_norm_residual from d_h_out [T, H] (the stream's type, or None) and d_x [T, H] (fp32, or None):
    d_h [T, H], d_y [T, H] (fp32, None without a branch) and each weight's gradient [H]."""
    lib = load()
    T, H = d_h.shape
    dev, f32, res = d_h.device, torch.float32, d_h.dtype
    ref = _norm_dtype(w_pre, w_post, gate)
    dt = res if ref is None else ref.dtype
    w = lambda t, name: _ptr(t, name, dt, (H,), dev)   # noqa: E731
    args = (_dt(d_h if ref is None else ref), _dt(d_h), _ptr(d_h_out, "d_h_out", res, (T, H), dev),
            _ptr(d_x, "d_x", f32, (T, H), dev), _ptr(h_out, "h_out", res, (T, H), dev),
            _ptr(rstd_pre, "rstd_pre", f32, (T,), dev), w(w_pre, "w_pre"), _ptr(y, "y", f32, (T, H), dev),
            _ptr(rstd_post, "rstd_post", f32, (T,), dev), w(w_post, "w_post"), w(gate, "gate"), T, H,
            float(weight_offset), float(residual_scale), float(branch_scale), _ptr(d_h, "d_h"),
            _ptr(d_y, "d_y", f32, (T, H), dev), w(d_w_pre, "d_w_pre"), w(d_w_post, "d_w_post"), w(d_gate, "d_gate"),
            _ptr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_norm_residual_backward, *args)


# Five steps of one quintic: singular values from about 0.01 of the largest on end between 0.68 and 1.13.
ORTHOGONAL_COEFS = ((3.4445, -4.7750, 2.0315),) * 5


def moe_orthogonal_update_workspace_bytes(dtype, out_dtype, batch, M, N, parts=1, has_momentum=False) -> int:
    return int(load().moe_orthogonal_update_workspace_bytes(_dtype_id(dtype), _dtype_id(out_dtype), int(batch), int(M),
                                                            int(N), int(parts), int(bool(has_momentum))))


def moe_orthogonal_update(grad, out, workspace, momentum=None, mu=0.95, nesterov=True, parts=1,
                          coefs=ORTHOGONAL_COEFS, eps=1e-7, scale=1.0, keep=0.0, stream=None):
    """out = keep out + scale orthogonalised(u), u the gradient or with ``momentum`` (fp32, in place) its step.  grad,
    momentum and out are [M, parts * N] or stacks [batch, M, parts * N] of matrices M x N, each orthogonalised by
    itself.  ``coefs``: (a, b, c) of every step."""
    lib = load()
    shape = grad.shape
    if len(shape) not in (2, 3):
        raise ValueError(f"grad must be a matrix or a stack of matrices (got shape {tuple(shape)})")
    batch, (M, N2) = (1 if len(shape) == 2 else shape[0]), shape[-2:]
    if parts < 1 or N2 % parts:
        raise ValueError(f"grad's {N2} columns are not {parts} matrices side by side")
    dev = grad.device
    coefs = [tuple(step) for step in coefs]
    if any(len(step) != 3 for step in coefs):
        raise ValueError("coefs must hold three numbers per step")
    flat = [float(v) for step in coefs for v in step]
    args = (_dt(grad), _dt(out), _ptr(grad, "grad"), _ptr(momentum, "momentum", torch.float32, shape, dev), float(mu),
            int(bool(nesterov)), batch, M, N2 // parts, int(parts), len(coefs),
            (_c_float * max(len(flat), 1))(*flat), float(eps), float(scale), float(keep),
            _ptr(out, "out", None, shape, dev), _ptr(workspace, "workspace", torch.uint8, None, dev),
            workspace.numel(), _stream(stream, dev))
    _call_on(dev, lib.moe_orthogonal_update, *args)


class MoEBlockBuffers:
    """Device buffers of a training step of a residual block around the layer for T tokens: the norms' outputs and
    factors, the router's losses, and the gradients of the stream and of the norms' weights.  ``stream_dtype`` is the
    residual stream's type, ``post_norm`` and ``gated_branch`` say whether the block norms the layer's output and
    gates it per channel."""

    def __init__(self, T, H, E, dtype, stream_dtype, device, post_norm=False, gated_branch=False):
        f32, i32 = torch.float32, torch.int32
        new = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)   # noqa: E731
        self.x, self.rstd_pre = new((T, H), dtype), new((T,), f32)
        self.h_out, self.rstd_post = new((T, H), stream_dtype), new((T,), f32) if post_norm else None
        self.losses, self.counts, self.tokens = new((2,), f32), new((E,), i32), new((1,), i32)
        self.prob_sums, self.lse = new((E,), f32), new((T,), f32)
        self.d_h, self.d_y = new((T, H), stream_dtype), new((T, H), f32)
        self.d_w_pre = new((H,), dtype)
        self.d_w_post = new((H,), dtype) if post_norm else None
        self.d_gate = new((H,), dtype) if gated_branch else None
        self.loss_ws = new((moe_balance_loss_workspace_bytes(T, E),), torch.uint8)
        with torch.cuda.device(device):   # the workspace goes by the device's compute units
            self.route_ws = new((moe_route_balance_backward_workspace_bytes(dtype, T, H, E, 1),), torch.uint8)
        self.norm_ws = new((moe_norm_residual_backward_workspace_bytes(T, H),), torch.uint8)
        self.norm, self.coef = new((1,), f32), new((1,), f32)
        self.grad_ws = new((moe_grad_norm_workspace_bytes(10),), torch.uint8)   # a layer's seven gradients, three here

    def grad_list(self, train):
        """The layer's gradients and the norms' as they are now, as one MoEGradList."""
        return MoEGradList(train.grad_tensors()
                           + [g for g in (self.d_w_pre, self.d_w_post, self.d_gate) if g is not None])


def moe_block_train_forward(h, w_pre, w_post, gate, w_router, logit_bias, W1, W2, top_k, shared, bufs, train, block,
                            token_mask=None, balance_coef=0.01, z_coef=0.0, eps=1e-6, weight_offset=0.0,
                            residual_scale=1.0, branch_scale=1.0, stream=None, layout=MOE_W_KN):
    """Training forward of h -> residual_scale h + branch_scale gate norm(layer(norm(h))) into block.h_out (``block`` a
    MoEBlockBuffers; w_post and gate may be None), with the router's losses in block.losses."""
    moe_norm_residual(h, None, None, None, w_pre, None, block.x, None, block.rstd_pre, eps, weight_offset,
                      stream=stream)
    moe_layer_train_forward(block.x, w_router, logit_bias, W1, W2, top_k, shared, bufs, train, stream, layout)
    moe_balance_loss(bufs.logits, bufs.topk_ids, token_mask, block.losses, block.counts, block.tokens,
                     block.prob_sums, block.lse, block.loss_ws, balance_coef, z_coef, stream)
    moe_norm_residual(h, bufs.y, w_post, gate, None, block.h_out, None, block.rstd_post, None, eps, weight_offset,
                      residual_scale, branch_scale, stream)
    return block.h_out


def moe_block_backward(d_h_out, h, w_pre, w_post, gate, w_router, W1, W2, shared, bufs, train, block, token_mask=None,
                       balance_coef=0.01, z_coef=0.0, weight_offset=0.0, residual_scale=1.0, branch_scale=1.0,
                       max_norm=None, stream=None, layout=MOE_W_KN):
    """Backward of moe_block_train_forward from d_h_out [T, H] (the stream's type) and of the sum of its losses:
    block.d_h, block.d_w_pre, block.d_w_post, block.d_gate and the layer's gradients in ``train``.  With ``max_norm``
    all parameters' gradients are scaled in place to at most that norm together (block.norm, block.coef).
    The stream's gradient rests in block.d_h between the two norms' calls, rounded to the stream's type: with a
    residual_scale of 1 that rounds nothing, with another one a bf16 stream's d_h takes a half step of its first term
    more than its own (a float32 array for it would cost its trip through memory)."""
    moe_norm_residual_backward(d_h_out, None, None, None, None, bufs.y, block.rstd_post, w_post, gate, block.d_h,
                               block.d_y, None, block.d_w_post, block.d_gate, block.norm_ws, weight_offset,
                               residual_scale, branch_scale, stream)
    moe_layer_backward(block.d_y, block.x, w_router, W1, W2, shared, bufs, train, None, stream, layout,
                       losses=MoERouteLosses(block, token_mask, balance_coef, z_coef))
    moe_norm_residual_backward(block.d_h, train.d_x, h, block.rstd_pre, w_pre, None, None, None, None, block.d_h,
                               None, block.d_w_pre, None, None, block.norm_ws, weight_offset, stream=stream)
    if max_norm is not None:
        grads = block.grad_list(train)
        moe_grad_norm(grads, block.norm, block.grad_ws, stream=stream)
        moe_grad_clip(grads, block.norm, max_norm, block.coef, stream=stream)
    return block


def _need_weights(w_router, W1, W2, shared, layout):
    """The layer's weights fit each other in this layout."""
    (H, E), nk = w_router.shape, layout == MOE_W_NK
    I = W2.shape[-1 if nk else -2]   # noqa: E741
    want = [("W1", W1, _w1_shape(E, H, I, layout)), ("W2", W2, _w2_shape(E, H, I, layout))]
    if shared is not None:
        I_s = shared[1].shape[-1 if nk else -2]
        want += [("ws1", shared[0], _ws1_shape(H, I_s, layout)), ("ws2", shared[1], _ws2_shape(H, I_s, layout))]
    for name, w, shape in want:
        if tuple(w.shape) != shape:
            raise ValueError(f"{name} must have shape {shape} in layout {'MOE_W_NK' if nk else 'MOE_W_KN'} beside the "
                             f"other weights (got {tuple(w.shape)})")


class MoEOrthogonalState:
    """Momenta (fp32) and workspace of moe_layer_orthogonal_step for the matrices of a layer: the experts' W1 and W2,
    the router's and the shared expert's weights (``shared`` as in moe_layer_train_forward, or None), of the types and
    layout in which the step updates them."""

    def __init__(self, w_router, W1, W2, shared=None, layout=MOE_W_KN):
        _need_weights(w_router, W1, W2, shared, layout)
        self.layout = layout
        weights = [W1, W2, w_router] + ([] if shared is None else [shared[0], shared[1]])
        self.momenta = [torch.zeros(w.shape, dtype=torch.float32, device=w.device) for w in weights]
        need = 0
        with torch.cuda.device(W1.device):   # the workspace goes by the device's compute units
            for w, fused in self._matrices(weights):
                shape, parts = self._split(w.shape, fused)
                batch = shape[0] if len(shape) == 3 else 1
                for grad in {w.dtype, torch.bfloat16}:   # float32 weights may have gradients of either type
                    need = max(need, moe_orthogonal_update_workspace_bytes(grad, w.dtype, batch, shape[-2],
                                                                           shape[-1] // parts, parts, True))
        self.ws = torch.empty((need,), dtype=torch.uint8, device=W1.device)

    @staticmethod
    def _matrices(weights):
        """(weight, whether it holds a gate and an up projection)."""
        return list(zip(weights, (True, False, False, True, False)))

    def _split(self, shape, fused):
        """(shape, parts) by which moe_orthogonal_update sees a weight: gate and up projections are matrices of
        their own, side by side in columns (MOE_W_KN) or one above the other."""
        if not fused:
            return tuple(shape), 1
        if self.layout == MOE_W_KN:
            return tuple(shape), 2
        batch = shape[0] if len(shape) == 3 else 1
        return (2 * batch, shape[-2] // 2, shape[-1]), 1


def moe_layer_orthogonal_step(w_router, W1, W2, shared, train, state, lr, mu=0.95, nesterov=True, weight_decay=0.0,
                              rms=0.2, coefs=ORTHOGONAL_COEFS, eps=1e-7, stream=None):
    """One step of the layer's matrices by their orthogonalised momentum, in place: for every M x N matrix w of W1
    (gate and up apart), W2, w_router, ws1 and ws2, w = (1 - lr weight_decay) w - lr rms sqrt(max(M, N)) X with X the
    orthogonalised momentum of its gradient in ``train`` (elements of X times sqrt(max(M, N)) have a root mean square
    of about 1).  ``state`` (MoEOrthogonalState) holds the momenta.  A bf16 weight keeps nothing of a step below half a
    step of its own (2^-9 to 2^-8 of it; a weight_decay lr of 0.001 alone changes none): for small rates give the step
    float32 copies of the weights, with their state, beside the bf16 gradients, and copy them into the layer's bf16
    weights after it (float32 results take three products for one)."""
    weights = [W1, W2, w_router] + ([] if shared is None else [shared[0], shared[1]])
    grads = [train.d_w1, train.d_w2, train.d_w_router] + ([] if shared is None else [train.d_ws1, train.d_ws2])
    if len(state.momenta) != len(weights):
        raise ValueError("the state was made for a layer with" + ("out" if shared is not None else "")
                         + " a shared expert")
    # all of them before the first update: a view below takes any shape of as many elements
    for name, w, g, m in zip(("W1", "W2", "w_router", "ws1", "ws2"), weights, grads, state.momenta):
        if g.shape != w.shape:
            raise ValueError(f"the training buffers' gradient of {name} has shape {tuple(g.shape)}, the weight "
                             f"{tuple(w.shape)}")
        if m.shape != w.shape:
            raise ValueError(f"the state was made for {name} of shape {tuple(m.shape)} (got {tuple(w.shape)})")
        _ptr(w, name, None, None, W1.device)
        _ptr(g, "the gradient of " + name, None, None, W1.device)
    for (w, fused), g, m in zip(state._matrices(weights), grads, state.momenta):
        shape, parts = state._split(w.shape, fused)
        scale = -lr * rms * max(shape[-2], shape[-1] // parts) ** 0.5
        moe_orthogonal_update(g.view(shape), w.view(shape), state.ws, m.view(shape), mu, nesterov, parts, coefs, eps,
                              scale, 1.0 - lr * weight_decay, stream)
