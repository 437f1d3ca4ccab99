"""GPU tests of the training calls at the edges of their ranges: values next to the types' limits, token counts next to
the launch limits, lists longer than a launch's table.  Bounds as in test_gpu_train: sums of K fp32 products within
4 (K + 16) 2^-24 of the magnitudes, half a step for a store."""

import numpy as np
import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B
from oracle import moe_oracle as O
from tests.test_gpu_train import DEV, TORCH, U, Out, check, dev

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
