"""GPU parity of the layer's training operators -- shared expert forward halves and backward halves, router backward,
gradient norm and clipping -- against the float64 oracle, element by element.

Bounds.  With u = 2^-24 (half a step of fp32) a sum of K products in fp32, in any order, is within about K u of the sum
of the products' magnitudes; 4 (K + 16) u covers it together with the handful of fp32 operations of an epilogue.  A
bf16 store adds at most half a step, 2^-8 of the value (2^-9 for most), and values that the oracle rounds to bf16 where
the kernels do (contract mode) are the same numbers on both sides.
"""

import numpy as np
import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B
from mixture_experts_ffn_05_amd import workloads as wl
from oracle import moe_oracle as O
from oracle import train_oracle as TO
from tests.gpu_helpers import assert_grad_close, host

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
LAYOUTS = [B.MOE_W_KN, B.MOE_W_NK]
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 64   # elements past every output that must stay as they were


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.load()


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dtype).to(DEV)


class Out:
    """An output tensor of NaN with a guard behind it."""

    def __init__(self, shape, dtype=torch.float32, fill=float("nan")):
        n = int(np.prod(shape))
        self.whole = torch.full((n + GUARD,), fill, dtype=dtype, device=DEV)
        self.whole[n:] = 7.0
        self.t = self.whole[:n].view(shape)

    def get(self):
        assert (self.whole[-GUARD:] == 7.0).all(), "wrote past the end"
        return host(self.t).astype(np.float64)


def check(got, want, bound, dtype, what):
    tol = bound + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else U * np.abs(want)) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside their bound, e.g. at "
                           f"{np.argwhere(bad)[0].tolist()}: {got[bad][0]} for {want[bad][0]} +- {tol[bad][0]:.3e}")


def acc(a, b):
    """Bound of fp32 sums a @ b (magnitudes)."""
    return 4 * (a.shape[1] + 16) * U * (np.abs(a) @ np.abs(b))


def draw_shared(T, H, I_s, dtype, gated, seed=0):
    rng = np.random.default_rng(1000 * seed + T + 7 * H + 13 * I_s)
    n = lambda *s: O.bf16_rne(rng.standard_normal(s).astype(np.float32)) if dtype == "bf16" else \
        rng.standard_normal(s).astype(np.float32)   # noqa: E731
    scale = lambda a, s: O.bf16_rne((a * np.float32(s)).astype(np.float32)) if dtype == "bf16" else \
        (a * np.float32(s)).astype(np.float32)   # noqa: E731
    p = {"x": n(T, H), "ws1": scale(n(H, 2 * I_s), H ** -0.5), "ws2": scale(n(I_s, H), I_s ** -0.5),
         "h_pre": n(T, 2 * I_s), "d_h": scale(n(T, 2 * I_s), 0.1),
         "dy": rng.standard_normal((T, H)).astype(np.float32),
         "y_shared": rng.standard_normal((T, H)).astype(np.float32),
         "d_z": rng.standard_normal(T).astype(np.float32), "gate": rng.uniform(0, 1, T).astype(np.float32),
         "w_gate": scale(n(H), H ** -0.5), "d_x0": rng.standard_normal((T, H)).astype(np.float32)}
    p["act"] = n(T, I_s)
    if not gated:
        for k in ("d_z", "gate", "w_gate", "y_shared"):
            p[k] = None
    return p


def stored(w, layout, dtype):
    return dev(w if layout == B.MOE_W_KN else w.T, TORCH[dtype])


def kn(w, layout):
    return w if layout == B.MOE_W_KN else w.T


# T, H, I_s: one row; fewer rows than any tile; one past a tile; several tiles; widths of one octet, of a part of a
# slice, of several slices and a tail; more reduction than output and the reverse
SIZES = [(1, 8, 8), (1, 256, 128), (2, 72, 40), (17, 8, 264), (63, 264, 8), (64, 64, 64), (65, 136, 200), (129, 320, 72),
         (200, 512, 264), (300, 128, 520), (517, 256, 136), (1030, 64, 128)]
SHARED = [(s, dt, g) for s in SIZES for dt, g in (("bf16", True), ("bf16", False))] + \
         [(s, "f32", True) for s in SIZES[1::2]] + [(SIZES[6], "f32", False)]
SHARED_IDS = [f"{'x'.join(map(str, s))}-{dt}{'-gated' if g else ''}" for s, dt, g in SHARED]


@pytest.mark.parametrize("layout", LAYOUTS, ids=["kn", "nk"])
@pytest.mark.parametrize("size,dtype,gated", SHARED, ids=SHARED_IDS)
def test_shared_forward(size, dtype, gated, layout):
    T, H, I_s = size
    print(f"[case] {size} {dtype} gated={gated} layout={layout}", flush=True)
    p = draw_shared(T, H, I_s, dtype, gated)
    td = TORCH[dtype]
    ws = torch.full((B.moe_shared_train_workspace_bytes(td, T, H, I_s),), 255, dtype=torch.uint8, device=DEV)
    act, h = Out((T, I_s), td), Out((T, 2 * I_s), td)
    x = dev(p["x"], td)
    B.moe_shared_fc1_save(x, stored(p["ws1"], layout, dtype), act.t, h.t, ws, layout=layout)
    torch.cuda.synchronize()
    a_ref, h_ref = TO.shared_fc1(p["x"], p["ws1"])
    hb = acc(p["x"].astype(np.float64), p["ws1"])
    check(h.get(), h_ref, hb, dtype, "h_pre")
    g, u = h_ref[:, :I_s], h_ref[:, I_s:]
    # |silu'| <= 1.1, |silu(g)| <= |g|; silu itself a few fp32 roundings
    check(act.get(), a_ref, 1.1 * hb[:, :I_s] * (np.abs(u) + hb[:, I_s:]) + np.abs(g) * hb[:, I_s:]
          + 16 * U * np.abs(a_ref), dtype, "act")

    for accumulate in (False, True):
        y = Out((T, H))
        y.t.copy_(dev(p["d_x0"]))
        ys, gate = (Out((T, H)), Out((T,))) if gated else (None, None)
        B.moe_shared_fc2_save(dev(p["act"], td), stored(p["ws2"], layout, dtype), x,
                              dev(p["w_gate"], td) if gated else None, y.t, ys.t if gated else None,
                              gate.t if gated else None, ws, accumulate=accumulate, layout=layout)
        torch.cuda.synchronize()
        y_ref, ys_ref, gate_ref = TO.shared_fc2(p["act"], p["ws2"], p["x"], p["w_gate"])
        yb = acc(p["act"].astype(np.float64), p["ws2"])
        if gated:
            check(ys.get(), ys_ref, yb, "f32", "y_shared")
            # sigmoid' <= 1/4 times the dot product's bound, and a few roundings
            zb = acc(p["x"].astype(np.float64), p["w_gate"][:, None])[:, 0]
            check(gate.get(), gate_ref, zb / 4 + 8 * U * gate_ref, "f32", "gate")
            yb = yb + np.abs(ys_ref) * (zb / 4 + 8 * U * gate_ref)[:, None]
        base = p["d_x0"].astype(np.float64) if accumulate else 0.0
        check(y.get(), y_ref + base, yb + 4 * U * (np.abs(y_ref) + np.abs(base)), "f32", "y")


@pytest.mark.parametrize("layout", LAYOUTS, ids=["kn", "nk"])
@pytest.mark.parametrize("size,dtype,gated", SHARED, ids=SHARED_IDS)
def test_shared_backward(size, dtype, gated, layout):
    T, H, I_s = size
    print(f"[case] {size} {dtype} gated={gated} layout={layout}", flush=True)
    p = draw_shared(T, H, I_s, dtype, gated, seed=1)
    td = TORCH[dtype]
    opt = lambda k, d=torch.float32: dev(p[k], d) if p[k] is not None else None   # noqa: E731
    ws = torch.full((B.moe_shared_train_workspace_bytes(td, T, H, I_s),), 255, dtype=torch.uint8, device=DEV)
    x, ws1, ws2 = dev(p["x"], td), stored(p["ws1"], layout, dtype), stored(p["ws2"], layout, dtype)

    d_h, d_ws2, d_z = Out((T, 2 * I_s), td), Out(tuple(ws2.shape), td), Out((T,)) if gated else None
    B.moe_shared_fc2_backward(dev(p["dy"]), dev(p["act"], td), dev(p["h_pre"], td), ws2, opt("y_shared"), opt("gate"),
                              d_h.t, d_ws2.t, d_z.t if gated else None, ws, layout=layout)
    torch.cuda.synchronize()
    contract = dtype == "bf16"
    dh_ref, dw_ref, dz_ref = TO.shared_fc2_backward(p["dy"], p["act"], p["h_pre"], p["ws2"], p["y_shared"], p["gate"],
                                                    contract=contract)
    D = p["dy"] if not gated else (p["dy"] * p["gate"][:, None]).astype(np.float32)
    D = (O.bf16_rne(D) if contract else D).astype(np.float64)
    dab = acc(D, p["ws2"].T.astype(np.float64))
    da = np.abs(D @ p["ws2"].T.astype(np.float64)) + dab
    g, u = p["h_pre"][:, :I_s].astype(np.float64), p["h_pre"][:, I_s:].astype(np.float64)
    s = 1 / (1 + np.exp(-g))
    # each factor's magnitude times the product's bound, and a few roundings of the epilogue's terms
    fg, fu = np.abs(u) * s * (1 + np.abs(g) * (1 - s)), np.abs(g) * s
    check(d_h.get(), dh_ref, np.concatenate([fg * (dab + 16 * U * da), fu * (dab + 16 * U * da)], axis=1), dtype, "d_h")
    check(kn(d_ws2.get(), layout), dw_ref, acc(p["act"].T.astype(np.float64), D), dtype, "d_ws2")
    if gated:
        mag = np.sum(np.abs(p["dy"].astype(np.float64) * p["y_shared"]), axis=1)
        check(d_z.get(), dz_ref, 4 * (H + 16) * U * mag * p["gate"] * (1 - p["gate"]) + 2 * U * np.abs(dz_ref), "f32",
              "d_gate_logit")

    for accumulate in (False, True):
        d_x, d_ws1, d_wg = Out((T, H)), Out(tuple(ws1.shape), td), Out((H,), td) if gated else None
        d_x.t.copy_(dev(p["d_x0"]))
        B.moe_shared_fc1_backward(dev(p["d_h"], td), x, ws1, opt("d_z"), opt("w_gate", td), d_x.t, d_ws1.t,
                                  d_wg.t if gated else None, ws, accumulate=accumulate, layout=layout)
        torch.cuda.synchronize()
        dx_ref, dw1_ref, dwg_ref = TO.shared_fc1_backward(p["d_h"], p["x"], p["ws1"], p["d_z"], p["w_gate"])
        base = p["d_x0"].astype(np.float64) if accumulate else 0.0
        rank1 = np.abs(np.outer(p["d_z"], p["w_gate"])) if gated else 0.0
        check(d_x.get(), dx_ref + base, acc(p["d_h"].astype(np.float64), p["ws1"].T) + 4 * U * (rank1 + np.abs(base)
              + np.abs(dx_ref)), "f32", "d_x")
        check(kn(d_ws1.get(), layout), dw1_ref, acc(p["x"].T.astype(np.float64), p["d_h"]), dtype, "d_ws1")
        if gated:
            check(d_wg.get(), dwg_ref, acc(p["x"].T.astype(np.float64), p["d_z"][:, None])[:, 0], dtype, "d_w_gate")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_saturated_gates(dtype):
    """Pre-activations far out on both sides: the sigmoid saturates to 0 and 1 without a NaN.  d_act is one column's
    dy times a weight of 1, so both halves of d_h have a closed form with a handful of roundings."""
    td = TORCH[dtype]
    T, H, I_s = 9, 8, 16
    g = np.array([0, 1, -1, 30, -30, 88, -88, 104, -104, 200, -200, 1e4, -1e4, 1e30, -1e30, -1e-30], np.float32)
    h = np.concatenate([np.tile(g, (T, 1)), np.full((T, I_s), 2.0, np.float32)], axis=1)
    h = O.bf16_rne(h) if dtype == "bf16" else h
    dy = np.zeros((T, H), np.float32)
    dy[:, 3] = 0.5
    ws2 = torch.zeros((I_s, H), dtype=td, device=DEV)
    ws2[:, 3] = 1.0
    d_h, d_ws2 = Out((T, 2 * I_s), td), Out((I_s, H), td)
    ws = torch.zeros((B.moe_shared_train_workspace_bytes(td, T, H, I_s),), dtype=torch.uint8, device=DEV)
    B.moe_shared_fc2_backward(dev(dy), torch.zeros((T, I_s), dtype=td, device=DEV), dev(h, td), ws2, None, None, d_h.t,
                              d_ws2.t, None, ws)
    torch.cuda.synchronize()
    z = h[:, :I_s].astype(np.float64)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-z))
    want = np.concatenate([0.5 * 2 * s * (1 + z * (1 - s)), 0.5 * z * s], axis=1)
    # s: a few ulp, or 0 where it is below the normal numbers (2^-126); 1 - s: an ulp of 1, and exactly 0 from z = 30 on,
    # where 1 + exp(-z) rounds to 1
    slack = np.where(z > 30, 0.0, U)
    mag = np.concatenate([s * (1 + np.abs(z) * (1 - s + slack)), np.abs(z) * s], axis=1)
    far = 2.0 ** -126 * np.concatenate([1 + np.abs(z), np.abs(z)], axis=1) * (np.tile(s, 2) < 1e-30)
    check(d_h.get(), want, 16 * U * mag + far, dtype, "d_h")


@pytest.mark.parametrize("layout", LAYOUTS, ids=["kn", "nk"])
@pytest.mark.parametrize("T,H,I_s,dtype", [(70, 136, 72, "bf16"), (300, 512, 640, "bf16"), (40, 72, 40, "f32")])
def test_a_row_that_is_not_finite_stays_in_its_row(T, H, I_s, dtype, layout):
    """One token's NaN or infinity reaches that token's rows only: outputs that mix no tokens are bit for bit what they
    are without it elsewhere."""
    p = draw_shared(T, H, I_s, dtype, True, seed=4)
    td, f32, bad = TORCH[dtype], torch.float32, T // 2
    ws = torch.zeros((B.moe_shared_train_workspace_bytes(td, T, H, I_s),), dtype=torch.uint8, device=DEV)
    ws1, ws2, wg = stored(p["ws1"], layout, dtype), stored(p["ws2"], layout, dtype), dev(p["w_gate"], td)
    new = lambda *s, dt=td: torch.zeros(s, dtype=dt, device=DEV)   # noqa: E731

    def run(v):
        x, act, dy = dev(p["x"], td), dev(p["act"], td), dev(p["dy"])
        dh_in, d_z = dev(p["d_h"], td), dev(p["d_z"])
        if v is not None:
            for t in (x, act, dy, dh_in):
                t[bad, 3] = v
        o = dict(act=new(T, I_s), h=new(T, 2 * I_s), y=new(T, H, dt=f32), ys=new(T, H, dt=f32), gate=new(T, dt=f32),
                 d_h=new(T, 2 * I_s), d_z=new(T, dt=f32), d_x=new(T, H, dt=f32))
        B.moe_shared_fc1_save(x, ws1, o["act"], o["h"], ws, layout=layout)
        B.moe_shared_fc2_save(act, ws2, x, wg, o["y"], o["ys"], o["gate"], ws, layout=layout)
        B.moe_shared_fc2_backward(dy, act, dev(p["h_pre"], td), ws2, dev(p["y_shared"]), dev(p["gate"]), o["d_h"],
                                  torch.empty_like(ws2), o["d_z"], ws, layout=layout)
        B.moe_shared_fc1_backward(dh_in, x, ws1, d_z, wg, o["d_x"], torch.empty_like(ws1), new(H), ws, layout=layout)
        torch.cuda.synchronize()
        return o

    want = run(None)
    keep = torch.arange(T, device=DEV) != bad
    for v in (float("nan"), float("inf")):
        got = run(v)
        for n in want:
            assert torch.equal(got[n][keep], want[n][keep]), (n, v)
            assert not torch.isfinite(got[n][bad]).all() or n == "gate", (n, v)


def draw_routes(T, E, k, seed):
    """Seeded routes: repeated experts, ids outside [0, E), an expert without tokens."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if E > 3:
        ids[ids == 2] = 1
    ids[0, :] = ids[0, 0]
    if T > 3:
        ids[2, 0], ids[3, k - 1] = -1, E
    w = rng.dirichlet(np.ones(k), T).astype(np.float32) if k > 1 else np.ones((T, 1), np.float32)
    return ids, w, (0.3 * rng.standard_normal((T, k))).astype(np.float32)


ROUTE = [(1, 8, 1, 1, "bf16"), (1, 256, 64, 6, "bf16"), (5, 72, 3, 2, "f32"), (17, 136, 60, 4, "bf16"),
         (130, 264, 7, 3, "bf16"), (128, 256, 8, 2, "f32"), (300, 512, 65, 8, "bf16"), (600, 128, 256, 8, "bf16"),
         (40, 64, 1024, 32, "bf16"), (33, 40, 1000, 5, "f32"), (1030, 2048, 64, 6, "bf16"), (90, 200, 4, 6, "bf16"),
         (2000, 24, 16, 1, "f32"), (150, 136, 1024, 32, "f32"), (70, 264, 1020, 32, "bf16")]


@pytest.mark.parametrize("case", ROUTE, ids=lambda c: "x".join(map(str, c)))
def test_route_backward(case):
    T, H, E, k, dtype = case
    print(f"[case] {case}", flush=True)
    rng = np.random.default_rng(T + E)
    td = TORCH[dtype]
    rnd = (lambda a: O.bf16_rne(a)) if dtype == "bf16" else (lambda a: a)
    x = rnd(rng.standard_normal((T, H)).astype(np.float32))
    wr = rnd((0.05 * rng.standard_normal((H, E))).astype(np.float32))
    ids, w, dw = draw_routes(T, E, k, T * E + k)
    dx0 = rng.standard_normal((T, H)).astype(np.float32)
    ws = torch.full((B.moe_route_backward_workspace_bytes(td, T, H, E, k),), 255, dtype=torch.uint8, device=DEV)
    dx_ref, dwr_ref, db_ref, dl = TO.route_backward(x, wr, ids, w, dw, contract=dtype == "bf16")
    mag = (np.abs(w) * (np.abs(dw) + np.sum(np.abs(w * dw), axis=1, keepdims=True))).astype(np.float64)
    dmag = np.zeros((T, E))      # magnitudes behind each logit's gradient, for the bound of its fp32 evaluation
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                dmag[t, ids[t, j]] += mag[t, j]
    dlb = 4 * (2 * k + 16) * U * dmag
    for accumulate, bias in ((False, True), (True, False)):
        d_x, d_wr, d_b = Out((T, H)), Out((H, E), td), Out((E,)) if bias else None
        d_x.t.copy_(dev(dx0))
        B.moe_route_backward(dev(x, td), dev(wr, td), torch.from_numpy(ids).to(DEV), dev(w), dev(dw), d_x.t, d_wr.t,
                             d_b.t if bias else None, ws, accumulate=accumulate)
        torch.cuda.synchronize()
        base = dx0.astype(np.float64) if accumulate else 0.0
        check(d_x.get(), dx_ref + base, dlb @ np.abs(wr.T).astype(np.float64)
              + 4 * (k + 16) * U * (dmag @ np.abs(wr.T) + np.abs(base)), "f32", "d_x")
        # a logit gradient whose fp32 value falls on the other side of a bf16 rounding border is off by a whole step,
        # 2^-7 of its value, and one within its own bound of zero by that bound
        flips = 2.0 ** -7 * np.abs(dl) + dlb if dtype == "bf16" else dlb
        near = np.abs(O.bf16_rne((dl + dlb).astype(np.float32)) - O.bf16_rne((dl - dlb).astype(np.float32))) > 0 \
            if dtype == "bf16" else np.ones_like(dl, bool)
        check(d_wr.get(), dwr_ref, np.abs(x.T).astype(np.float64) @ (flips * near)
              + acc(np.abs(x.T).astype(np.float64), np.abs(dl)), dtype, "d_w_router")
        if bias:
            check(d_b.get(), db_ref, dlb.sum(axis=0) + 4 * (T + 16) * U * dmag.sum(axis=0), "f32", "d_logit_bias")
    if E > 3:
        assert not d_wr.get()[:, 2].any()   # an expert without tokens: a gradient of zeros, written


# ------------------------------------------------------------------------------------------
# norm and clipping
# ------------------------------------------------------------------------------------------
def grad_list(sizes, offsets=None, seed=3, std=1.0):
    """bf16 and fp32 tensors cut out of two buffers at the given offsets (elements)."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = torch.bfloat16 if i % 3 else torch.float32
        off = 0 if offsets is None else offsets[i % len(offsets)]
        buf = torch.randn((n + off + GUARD,), generator=g).mul_(std).to(dt).to(DEV)
        out.append(buf[off:off + n])
    return out


def norm_of(grads):
    n = torch.full((1,), -1.0, device=DEV)
    sq = torch.full((1,), -1.0, dtype=torch.float64, device=DEV)
    lst = B.MoEGradList(grads)
    ws = torch.full((B.moe_grad_norm_workspace_bytes(lst.n),), 255, dtype=torch.uint8, device=DEV)
    B.moe_grad_norm(lst, n, ws, sum_sq=sq)
    torch.cuda.synchronize()
    return n, float(sq)


LISTS = {"one": ([1], None), "sizes": ([0, 1, 2, 7, 8, 9, 255, 16383, 16384, 16385, 40000, 0, 3], None),
         "off": ([5, 17, 1000, 16390, 33000, 4, 8, 1, 0], [1, 3, 5, 2, 7]), "many": (list(range(1, 260)), [0, 1]),
         "batches": ([40000] * 230, None)}


@pytest.mark.parametrize("name", LISTS)
def test_grad_norm_and_clip(name):
    print(f"[case] {name}", flush=True)
    sizes, offs = LISTS[name]
    grads = grad_list(sizes, offs)
    h = [host(g).astype(np.float64) for g in grads]
    want = TO.grad_norm(h)
    n, sq = norm_of(grads)
    # the sum of squares is fp64 on both sides; the norm is rounded to fp32 once
    assert abs(sq - want ** 2) <= 1e-10 * want ** 2
    assert abs(float(n) - want) <= 2 * U * want
    for max_norm in (0.37 * want, 0.0):
        c_ref = TO.clip_coef(float(n), np.float32(max_norm).item())
        outs = [Out((g.numel(),), g.dtype) for g in grads]
        coef = torch.full((1,), -1.0, device=DEV)
        B.moe_grad_clip(B.MoEGradList(grads, [o.t for o in outs]), n, max_norm, coef)
        torch.cuda.synchronize()
        assert abs(float(coef) - c_ref) <= 2 * U * c_ref
        for g, v, o in zip(grads, h, outs):
            check(o.get(), v * float(coef), U * np.abs(v * c_ref), "bf16" if g.dtype == torch.bfloat16 else "f32", name)
            np.testing.assert_array_equal(host(g).astype(np.float64), v)   # the input stays
    # in place: the same bits as out of place
    c_in = torch.full((1,), -1.0, device=DEV)
    outs = [torch.empty_like(g) for g in grads]
    B.moe_grad_clip(B.MoEGradList(grads, outs), n, 0.37 * want)
    B.moe_grad_clip(B.MoEGradList(grads), n, 0.37 * want, c_in)
    torch.cuda.synchronize()
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)


def test_grad_clip_below_the_norm_changes_nothing():
    grads = grad_list([10, 20000, 7], [1, 2])
    keep = [g.clone() for g in grads]
    n, _ = norm_of(grads)
    outs = [torch.zeros_like(g) for g in grads]
    coef = torch.zeros((1,), device=DEV)
    B.moe_grad_clip(B.MoEGradList(grads), n, 2 * float(n), coef)
    B.moe_grad_clip(B.MoEGradList(grads, outs), n, 2 * float(n))
    torch.cuda.synchronize()
    assert float(coef) == 1.0
    for g, k, o in zip(grads, keep, outs):
        assert torch.equal(g, k) and torch.equal(o, k)


def test_grad_clip_misaligned_outputs():
    """Inputs and outputs whose alignments differ, and outputs of another shape."""
    src = grad_list([33000, 33001, 4097], [1, 2, 0])
    big = [torch.zeros((g.numel() + 8,), dtype=g.dtype, device=DEV) for g in src]
    outs = [b[k:k + g.numel()] for b, g, k in zip(big, src, (2, 1, 3))]
    n, _ = norm_of(src)
    B.moe_grad_clip(B.MoEGradList(src, outs), n, 0.5 * float(n))
    torch.cuda.synchronize()
    c = TO.clip_coef(float(n), np.float32(0.5 * float(n)).item())
    for g, o, b, k in zip(src, outs, big, (2, 1, 3)):
        v = host(g).astype(np.float64) * c
        check(host(o).astype(np.float64), v, 4 * U * np.abs(v), "bf16" if g.dtype == torch.bfloat16 else "f32", "out")
        assert not b[:k].any() and not b[k + g.numel():].any()


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 3e38, 1e-38])
def test_grad_norm_of_extreme_values(value):
    """Squares that leave fp32's range in either direction, and values that are not finite."""
    grads = [torch.full((5,), value, device=DEV), torch.zeros((300,), dtype=torch.bfloat16, device=DEV)]
    n, sq = norm_of(grads)
    got = float(n)
    if np.isfinite(value):
        v = float(grads[0][0])
        want = np.sqrt(5) * v
        assert abs(sq - 5 * v * v) <= 1e-12 * 5 * v * v
        assert (got == np.inf) if want > 3.4028235e38 else abs(got - want) <= 2 * U * want
        if got == np.inf:
            return
    coef = torch.zeros((1,), device=DEV)
    outs = [torch.zeros_like(g) for g in grads]
    B.moe_grad_clip(B.MoEGradList(grads, outs), n, 1.0, coef)
    torch.cuda.synchronize()
    if np.isnan(value):
        assert np.isnan(got) and np.isnan(float(coef)) and outs[0].isnan().all() and outs[1].isnan().all()
    elif np.isinf(value):
        assert got == np.inf and float(coef) == 0.0 and outs[0].isnan().all() and not outs[1].any()
    else:
        assert float(coef) == np.float32(TO.clip_coef(got, 1.0))


def test_grad_norm_past_two_to_the_31_elements():
    """One tensor of more than 2^31 elements: a few values far apart decide the norm."""
    n = (1 << 31) + 16384 + 5
    g = torch.zeros((n,), dtype=torch.bfloat16, device=DEV)
    at = [0, 12345, (1 << 31) - 1, 1 << 31, n - 6, n - 1]
    for i, k in enumerate(at):
        g[k] = float(2 ** i)
    lst = B.MoEGradList([g])
    norm = torch.zeros((1,), device=DEV)
    ws = torch.empty((B.moe_grad_norm_workspace_bytes(1),), dtype=torch.uint8, device=DEV)
    B.moe_grad_norm(lst, norm, ws)
    B.moe_grad_clip(lst, norm, 1.0)
    torch.cuda.synchronize()
    want = np.sqrt(sum(4.0 ** i for i in range(len(at))))
    assert abs(float(norm) - want) <= 2 * U * want
    for i, k in enumerate(at):
        assert abs(float(g[k]) - 2 ** i / want) <= 2.0 ** -8 * 2 ** i / want
    assert int(torch.count_nonzero(g[: 1 << 30])) == 2


# ------------------------------------------------------------------------------------------
# the operators together
# ------------------------------------------------------------------------------------------
LAYERS = [wl.LayerConfig("train_gated_bf16", "bf16", T=150, H=256, E=12, top_k=3, I=128, I_s=136, gated=True),
          wl.LayerConfig("train_bf16", "bf16", T=70, H=192, E=8, top_k=2, I=64, I_s=320),
          wl.LayerConfig("train_gated_f32", "f32", T=40, H=64, E=6, top_k=2, I=32, I_s=48, gated=True, fan_in_init=True),
          wl.LayerConfig("train_routed_only_f32", "f32", T=33, H=64, E=5, top_k=2, I=32, fan_in_init=True)]


def layer_step(cfg, layout, layer, dy, bias, max_norm=None, stream=None, bufs=None, train=None):
    dt = TORCH["bf16" if cfg.dtype == "bf16" else "f32"]
    t = (lambda w: w) if layout == B.MOE_W_KN else (lambda w: w.transpose(-1, -2).contiguous())
    W1, W2 = t(layer["W1"]), t(layer["W2"])
    sh = layer["shared"]
    shared = None if sh is None else (t(sh[0]), t(sh[1]), sh[2])
    bufs = bufs or B.MoELayerBuffers(cfg.T, cfg.H, cfg.E, cfg.top_k, cfg.I, cfg.I_s, dt, DEV)
    train = train or B.MoETrainBuffers(cfg.T, cfg.H, cfg.E, cfg.top_k, cfg.I, cfg.I_s, cfg.gated, True, dt, DEV, layout)
    B.moe_layer_train_forward(layer["x"], layer["w_router"], bias, W1, W2, cfg.top_k, shared, bufs, train, stream, layout)
    B.moe_layer_backward(dy, layer["x"], layer["w_router"], W1, W2, shared, bufs, train, max_norm, stream, layout)
    return bufs, train


@pytest.mark.parametrize("layout", LAYOUTS, ids=["kn", "nk"])
@pytest.mark.parametrize("cfg", LAYERS, ids=lambda c: c.name)
def test_layer_training_step(cfg, layout):
    """Forward, backward and clipping of a whole layer against the oracle's layer for the same routes."""
    print(f"[case] {cfg.name} layout={layout}", flush=True)
    layer = wl.make_layer(cfg, DEV)
    dy = np.random.default_rng(4).standard_normal((cfg.T, cfg.H)).astype(np.float32)
    bias = dev(np.linspace(-0.2, 0.2, cfg.E))
    bufs, tr = layer_step(cfg, layout, layer, dev(dy), bias)
    torch.cuda.synchronize()
    x, W1, W2, wr = host(layer["x"]), host(layer["W1"]), host(layer["W2"]), host(layer["w_router"])
    ids, w = host(bufs.topk_ids), host(bufs.topk_weights)
    contract = cfg.dtype == "bf16"
    ref = O.moe_backward(x, list(W1), list(W2), (ids, w), dy, contract=contract)
    dx_r, dwr, db, _ = TO.route_backward(x, wr, ids, w, ref["dweights"], contract)
    want = {"d_w1": ref["dW1"], "d_w2": ref["dW2"], "d_w_router": dwr, "d_logit_bias": db}
    d_x = ref["dx"] + dx_r
    y = O.moe_forward(x, None, list(W1), list(W2), cfg.top_k, routes=(ids, w), contract=contract)["y"]
    if cfg.I_s:
        ws1, ws2 = host(layer["shared"][0]), host(layer["shared"][1])
        wg = host(layer["shared"][2]) if cfg.gated else None
        rnd = O.bf16_rne if contract else (lambda a: a)
        act, h = TO.shared_fc1(x, ws1)
        act, h = rnd(act.astype(np.float32)), rnd(h.astype(np.float32))
        ysum, ys, gate = TO.shared_fc2(act, ws2, x, wg)
        y = y + ysum
        d_h, dw2s, dz = TO.shared_fc2_backward(dy, act, h, ws2, ys, gate, contract)
        dxs, dw1s, dwg = TO.shared_fc1_backward(rnd(d_h.astype(np.float32)), x, ws1, dz, wg)
        d_x = d_x + dxs
        want |= {"d_ws1": dw1s, "d_ws2": dw2s}
        if cfg.gated:
            want["d_w_gate"] = dwg
    assert_grad_close(host(bufs.y), y, cfg.dtype, "y")
    assert_grad_close(host(tr.d_x), d_x, cfg.dtype, "d_x")
    for name, ref_g in want.items():
        got = host(getattr(tr, name))
        if layout == B.MOE_W_NK and name in ("d_w1", "d_w2", "d_ws1", "d_ws2"):
            got = np.swapaxes(got, -1, -2)
        assert_grad_close(got, ref_g, cfg.dtype, name)
    # clipping, in place, to a third of the norm
    before = {n: host(getattr(tr, n)).astype(np.float64) for n in want}
    norm = TO.grad_norm(before.values())
    B.moe_grad_norm(tr.grads, tr.norm, tr.norm_ws)
    B.moe_grad_clip(tr.grads, tr.norm, norm / 3, tr.coef)
    torch.cuda.synchronize()
    assert abs(float(tr.norm) - norm) <= 2 * U * norm
    for n, v in before.items():
        got = getattr(tr, n)
        check(host(got).astype(np.float64), v * float(tr.coef), 0.0,
              "bf16" if got.dtype == torch.bfloat16 else "f32", n)


def test_layer_gradients_match_differences():
    """Central differences of the float32 layer's own forward along random directions.  y is computed to about 1e-6 of
    its size, so with a step of 1e-2 a difference is good to about 1e-4 of the gradient's size from rounding and
    h^2 = 1e-4 from truncation; routes are held fixed by a bias that separates the experts."""
    cfg = LAYERS[2]
    layer = wl.make_layer(cfg, DEV)
    rng = np.random.default_rng(11)
    dy = rng.standard_normal((cfg.T, cfg.H)).astype(np.float32)
    bias = dev(np.array([30.0, 29.5, 0, -1, -2, -3])[: cfg.E])    # experts 0 and 1 for every token
    layer["w_router"] = layer["w_router"] * 0.05
    bufs, tr = layer_step(cfg, B.MOE_W_KN, layer, dev(dy), bias)
    torch.cuda.synchronize()
    ids0 = host(bufs.topk_ids).copy()
    ws1, ws2, wg = layer["shared"]
    params = {"d_x": layer["x"], "d_w_router": layer["w_router"], "d_w1": layer["W1"], "d_w2": layer["W2"],
              "d_ws1": ws1, "d_ws2": ws2, "d_w_gate": wg, "d_logit_bias": bias}
    grads = {n: host(getattr(tr, n)).astype(np.float64).copy() for n in params}
    h = 1e-2
    for name, p in params.items():
        d = rng.standard_normal(tuple(p.shape)).astype(np.float32)
        d /= np.linalg.norm(d)
        keep, loss = p.clone(), []
        for sgn in (1, -1):
            p.copy_(keep + sgn * h * dev(d))
            b, _ = layer_step(cfg, B.MOE_W_KN, layer, dev(dy), bias)
            torch.cuda.synchronize()
            assert sorted(set(map(tuple, np.sort(host(b.topk_ids), axis=1)))) == \
                sorted(set(map(tuple, np.sort(ids0, axis=1))))
            loss.append(np.sum(dy.astype(np.float64) * host(b.y)))
        p.copy_(keep)
        fd = (loss[0] - loss[1]) / (2 * h)
        an = float(np.sum(grads[name] * d))
        scale = np.linalg.norm(grads[name])
        assert abs(fd - an) <= 2e-3 * scale + 2e-3, f"{name}: {fd} against {an} (|g| {scale})"


def test_layer_step_on_another_stream_and_as_a_graph():
    """The whole step, clipping included, on a side stream and captured into a graph: replays with new inputs, with
    eager work between them, equal the eager results bit for bit."""
    cfg = LAYERS[0]
    layer = wl.make_layer(cfg, DEV)
    bias = dev(np.linspace(-0.2, 0.2, cfg.E))
    rng = np.random.default_rng(12)
    inputs = [(dev(rng.standard_normal((cfg.T, cfg.H)), torch.bfloat16), dev(rng.standard_normal((cfg.T, cfg.H))))
              for _ in range(4)]
    names = ("d_x", "d_w1", "d_w2", "d_ws1", "d_ws2", "d_w_gate", "d_w_router", "d_logit_bias", "norm", "coef")

    def eager(x, dy):
        b, t = layer_step(cfg, B.MOE_W_KN, {**layer, "x": x}, dy, bias, max_norm=0.5)
        torch.cuda.synchronize()
        return [b.y.clone()] + [getattr(t, n).clone() for n in names]

    want = [eager(x, dy) for x, dy in inputs]
    x, dy = inputs[0][0].clone(), inputs[0][1].clone()
    sh = {**layer, "x": x}
    td = torch.bfloat16
    bufs = B.MoELayerBuffers(cfg.T, cfg.H, cfg.E, cfg.top_k, cfg.I, cfg.I_s, td, DEV)
    tr = B.MoETrainBuffers(cfg.T, cfg.H, cfg.E, cfg.top_k, cfg.I, cfg.I_s, cfg.gated, True, td, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer_step(cfg, B.MOE_W_KN, sh, dy, bias, 0.5, side, bufs, tr)
    side.synchronize()
    for n, w in zip(("y",) + names, want[0]):
        assert torch.equal(bufs.y if n == "y" else getattr(tr, n), w), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer_step(cfg, B.MOE_W_KN, sh, dy, bias, 0.5, None, bufs, tr)
    for r in range(2):
        for (xi, dyi), w in zip(inputs, want):
            x.copy_(xi)
            dy.copy_(dyi)
            graph.replay()
            torch.cuda.synchronize()
            for n, v in zip(("y",) + names, w):
                assert torch.equal(bufs.y if n == "y" else getattr(tr, n), v), (r, n)
            torch.randn((1000,), device=DEV).sum().item()


def test_two_layer_steps_at_once():
    """Two steps with their own buffers on two streams, their launches interleaved: each gives what it gives alone."""
    cfgs = [LAYERS[0], LAYERS[1]]
    names = ("d_x", "d_w1", "d_w2", "d_w_router", "d_logit_bias", "norm", "coef")
    problems = []
    for i, cfg in enumerate(cfgs):
        rng = np.random.default_rng(30 + i)
        layer = wl.make_layer(cfg, DEV)
        problems.append((cfg, layer, dev(rng.standard_normal((cfg.T, cfg.H))), dev(np.linspace(-0.3, 0.3, cfg.E))))
    want, held = [], []
    for cfg, layer, dy, bias in problems:
        held.append(layer_step(cfg, B.MOE_W_KN, layer, dy, bias, max_norm=0.1))
        b, t = held[-1]
        want.append([b.y.clone()] + [getattr(t, n).clone() for n in names])
        for v in (b.y, *(getattr(t, n) for n in names)):
            v.fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in cfgs]
    torch.cuda.synchronize()
    for _ in range(5):
        for (cfg, layer, dy, bias), s, (b, t) in zip(problems, streams, held):
            layer_step(cfg, B.MOE_W_KN, layer, dy, bias, 0.1, s, b, t)
        torch.cuda.synchronize()
        for (b, t), w in zip(held, want):
            for n, v in zip(("y",) + names, w):
                assert torch.equal(b.y if n == "y" else getattr(t, n), v), n


def test_refusals_on_device_tensors():
    """The binding's own checks: types, shapes, layouts, alignment, overlapping outputs."""
    T, H, I = 4, 16, 8
    bf = torch.bfloat16
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt, device=DEV)   # noqa: E731
    ws = torch.zeros((B.moe_shared_train_workspace_bytes(bf, T, H, I),), dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        B.moe_shared_fc1_save(z(T, H), z(H, I), z(T, I), z(T, 2 * I), ws)
    with pytest.raises(TypeError):
        B.moe_shared_fc1_save(z(T, H), z(H, 2 * I), z(T, I, dt=torch.float32), z(T, 2 * I), ws)
    with pytest.raises(ValueError):
        B.moe_shared_fc1_save(z(H, T).t(), z(H, 2 * I), z(T, I), z(T, 2 * I), ws)     # not contiguous
    with pytest.raises(B.MoEError, match="aligned"):
        B.moe_shared_fc1_save(z(T * H + 1)[1:].view(T, H), z(H, 2 * I), z(T, I), z(T, 2 * I), ws)
    with pytest.raises(B.MoEError, match="workspace needs"):
        B.moe_shared_fc2_backward(z(T, H, dt=torch.float32), z(T, I), z(T, 2 * I), z(I, H), None, None, z(T, 2 * I),
                                  z(I, H), None, ws[:16])
    with pytest.raises(B.MoEError, match="y_shared must not be NULL"):
        B.moe_shared_fc2_save(z(T, I), z(I, H), z(T, H), z(H), z(T, H, dt=torch.float32), None, None, ws)
    with pytest.raises(B.MoEError, match="y_shared must be NULL"):
        B.moe_shared_fc2_save(z(T, I), z(I, H), z(T, H), None, z(T, H, dt=torch.float32), z(T, H, dt=torch.float32),
                              None, ws)
    with pytest.raises(ValueError):
        B.MoEGradList([])
    with pytest.raises(TypeError):
        B.MoEGradList([torch.zeros(4, dtype=torch.float16, device=DEV)])
    with pytest.raises(ValueError):
        B.MoEGradList([z(4)], [z(5)])
    with pytest.raises(ValueError):
        B.MoEGradList([torch.zeros(4)])
    a = z(64, dt=torch.float32)
    n = torch.ones((1,), device=DEV)
    with pytest.raises(B.MoEError, match="overlaps"):
        B.moe_grad_clip(B.MoEGradList([a, a]), n, 1.0)
    with pytest.raises(B.MoEError, match="overlaps"):
        B.moe_grad_clip(B.MoEGradList([a[:32], a[32:]], [a[8:40], z(32, dt=torch.float32)]), n, 1.0)
    with pytest.raises(B.MoEError, match="max_norm"):
        B.moe_grad_clip(B.MoEGradList([a]), n, float("nan"))
    assert not a.any()
