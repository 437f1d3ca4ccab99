"""Cases and plain forms of the operators that train a whole MoE FFN layer.

The layer's routed experts have a backward pass of their own; these operators are what a training step of the layer
needs next to it:

* the shared expert (a gated feed-forward block) in training: ``fc1`` keeps its pre-activation, ``fc2`` keeps the
  ungated output and the gate, and each half has its backward call, the sigmoid gate's gradient included;
* the router's backward: through the softmax over the selected logits into x, the router weight and the logit bias;
* the norm of all of the layer's gradients together, and the gradients scaled to at most a given norm.

Weights are stored as the layer stores them: "kn" is [K, N] (x @ W), "nk" is [N, K].
"""

import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DEV = "cuda"


def _case(name, op, **kw):
    return {"name": name, "op": op, **kw}


def listed():
    return [
        # one small micro-batch of the DeepSeek-V2-Lite-shaped shared expert (two experts stored as one MLP)
        _case("fc1_save_v2l_t64", "fc1_save", T=64, H=2048, I_s=2816, dt=BF16, layout="kn"),
        # its training prefill
        _case("fc1_save_v2l", "fc1_save", T=8192, H=2048, I_s=2816, dt=BF16, layout="kn"),
        # a ragged batch of the Qwen2-MoE-shaped shared expert, gated, weights as a linear layer stores them
        _case("fc2_save_qwen2_t1021", "fc2_save", T=1021, H=2048, I_s=5632, dt=BF16, layout="nk", gated=True),
        # the widest shared expert, ungated (Llama-4-Scout-shaped)
        _case("fc2_save_scout", "fc2_save", T=2048, H=5120, I_s=8192, dt=BF16, layout="kn", gated=False),
        # a short ragged batch, ungated
        _case("fc2_bwd_v2l_t517", "fc2_bwd", T=517, H=2048, I_s=2816, dt=BF16, layout="nk", gated=False),
        # the gated shared expert's training batch
        _case("fc2_bwd_qwen2", "fc2_bwd", T=4096, H=2048, I_s=5632, dt=BF16, layout="kn", gated=True),
        # the float32 correctness workload: launches and latency
        _case("fc1_bwd_tiny_f32", "fc1_bwd", T=128, H=256, I_s=128, dt=F32, layout="kn", gated=True),
        # the largest product: input, weight and gate gradients of the gated gate/up projection
        _case("fc1_bwd_qwen2", "fc1_bwd", T=4096, H=2048, I_s=5632, dt=BF16, layout="kn", gated=True),
        # 60 experts, an odd number of tokens
        _case("route_bwd_qwen2_t1021", "route_bwd", T=1021, H=2048, E=60, top_k=4, dt=BF16, bias=False),
        # 256 experts with a logit bias, a full training batch
        _case("route_bwd_v3", "route_bwd", T=4096, H=7168, E=256, top_k=8, dt=BF16, bias=True),
        # a model's worth of small tensors (norm weights, biases, small projections) of both types, odd sizes, packed
        # one behind the other so that most start off any alignment
        _case("clip_many_ragged", "grad_clip", shapes="many", n=300, most=400_000, max_norm=1.0),
        # all gradients of a DeepSeek-V2-Lite-shaped layer: 64 experts, shared expert, router
        _case("clip_v2l_layer", "grad_clip", shapes="layer", H=2048, E=64, I=1408, I_s=2816, max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fc1_save", "fc2_save", "fc2_bwd", "fc1_bwd", "route_bwd", "grad_clip"])
    if op == "grad_clip":
        max_norm = rng.choice([0.1, 1.0, 1e6])
        if rng.random() < 0.5:
            return {"op": op, "shapes": "many", "n": _log_int(rng, 1, 400), "most": _log_int(rng, 10, 1_000_000),
                    "max_norm": max_norm}
        return {"op": op, "shapes": "layer", "H": 8 * _log_int(rng, 32, 256), "E": _log_int(rng, 4, 64),
                "I": 8 * _log_int(rng, 16, 176), "I_s": 8 * _log_int(rng, 16, 352), "max_norm": max_norm}
    dt = BF16 if rng.random() < 0.85 else F32
    if op == "route_bwd":
        E = _log_int(rng, 4, 256)
        return {"op": op, "T": _log_int(rng, 1, 4096 if dt == BF16 else 1024), "H": 8 * _log_int(rng, 32, 896), "E": E,
                "top_k": min(E, rng.randint(1, 8)), "dt": dt, "bias": rng.random() < 0.5}
    layout = rng.choice(["kn", "nk"])
    if dt == F32:
        case = {"op": op, "T": _log_int(rng, 1, 256), "H": 8 * _log_int(rng, 8, 64), "I_s": 8 * _log_int(rng, 8, 32)}
    else:
        # widths in steps of 64 as models have them, one in four in steps of 8
        step = 8 if rng.random() < 0.25 else 64
        H = step * _log_int(rng, 256 // step, 5120 // step)
        I_s = step * _log_int(rng, 128 // step, 8192 // step)
        T = _log_int(rng, 1, min(8192, 47_000_000_000 // (H * I_s)))
        case = {"op": op, "T": T, "H": H, "I_s": I_s}
    case |= {"dt": dt, "layout": layout}
    return case if op == "fc1_save" else case | {"gated": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dt"] == BF16 else torch.float32


def _shape(case, k, n):
    """Shape of a weight of k inputs and n outputs."""
    return (k, n) if case["layout"] == "kn" else (n, k)


def _kn(case, w):
    """A weight as its [K, N] matrix."""
    return w if case["layout"] == "kn" else w.t()


def _split(h):
    half = h.shape[-1] // 2
    return h[..., :half], h[..., half:]


def _numels(case, seed):
    """[(number of elements, type)] of a gradient list."""
    if case["shapes"] == "layer":
        H, E, I, I_s = (case[k] for k in ("H", "E", "I", "I_s"))
        return [(n, torch.bfloat16) for n in (E * H * 2 * I, E * I * H, H * 2 * I_s, I_s * H, H * E)]
    g = torch.Generator().manual_seed(12345 + case["n"] + case["most"])
    u = torch.rand((case["n"],), generator=g, dtype=torch.float64)
    sizes = torch.exp(u * math.log(case["most"])).long().clamp(1).tolist()
    kinds = (torch.rand((case["n"],), generator=g) < 0.7).tolist()
    return [(n, torch.bfloat16 if b else torch.float32) for n, b in zip(sizes, kinds)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(shape, std, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op == "grad_clip":
        lists = _numels(case, seed)
        flats, outs = {}, {}
        for dtype in (torch.bfloat16, torch.float32):
            total = sum(n for n, d in lists if d == dtype)
            flats[dtype] = torch.empty((total,), dtype=dtype, device=DEV)
            for i in range(0, total, 1 << 27):
                part = flats[dtype][i:i + (1 << 27)]
                part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * 1e-2)
            outs[dtype] = torch.zeros_like(flats[dtype])
        s["grads"], s["outs"], at = [], [], {torch.bfloat16: 0, torch.float32: 0}
        for n, d in lists:
            s["grads"].append(flats[d][at[d]:at[d] + n])
            s["outs"].append(outs[d][at[d]:at[d] + n])
            at[d] += n
        s["flat_outs"] = [o for o in outs.values() if o.numel()]
        s["norm"] = torch.zeros((1,), device=DEV)
        s["coef"] = torch.zeros((1,), device=DEV)
        if own:
            from mixture_experts_ffn_05_amd import binding as B
            s["plan"] = B.MoEGradList(s["grads"], s["outs"])
            s["ws"] = torch.empty((B.moe_grad_norm_workspace_bytes(len(lists)),), dtype=torch.uint8, device=DEV)
        return s

    dtype = _dtype(case)
    T, H = case["T"], case["H"]
    if op == "route_bwd":
        E, k = case["E"], case["top_k"]
        s["x"] = normal((T, H), 1.0, dtype)
        s["w_router"] = normal((H, E), 0.02, dtype)
        # a few experts are favoured, as in trained routers
        logits = normal((T, E), 0.9) + normal((E,), 0.7)
        top, ids = logits.topk(k, dim=1)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["weights"] = torch.softmax(top, dim=1).contiguous()
        s["d_weights"] = normal((T, k), 0.05)
        s["d_x"] = normal((T, H), 0.02)          # what the experts' backward left there
        s["d_w_router"] = torch.zeros((H, E), dtype=dtype, device=DEV)
        s["d_bias"] = torch.zeros((E,), device=DEV) if case["bias"] else None
        if own:
            from mixture_experts_ffn_05_amd import binding as B
            s["ws"] = torch.empty((B.moe_route_backward_workspace_bytes(dtype, T, H, E, k),), dtype=torch.uint8,
                                  device=DEV)
        return s

    I_s = case["I_s"]
    gated = case.get("gated", False)
    if op == "fc1_save":
        s["x"] = normal((T, H), 1.0, dtype)
        s["ws1"] = normal(_shape(case, H, 2 * I_s), 0.02, dtype)
        s["act"] = torch.zeros((T, I_s), dtype=dtype, device=DEV)
        s["h_pre"] = torch.zeros((T, 2 * I_s), dtype=dtype, device=DEV)
    else:
        s["x"] = normal((T, H), 1.0, dtype)
    s["w_gate"] = normal((H,), 0.02, dtype) if gated else None
    if op in ("fc2_save", "fc2_bwd"):
        s["h_pre"] = normal((T, 2 * I_s), 0.02 * math.sqrt(H), dtype)
        g, u = _split(s["h_pre"].float())
        s["act"] = (g / (1 + torch.exp(-g)) * u).to(dtype)
        s["ws2"] = normal(_shape(case, I_s, H), 0.02, dtype)
    if op == "fc2_save":
        s["y"] = torch.zeros((T, H), device=DEV)
        s["y_shared"] = torch.zeros((T, H), device=DEV) if gated else None
        s["gate"] = torch.zeros((T,), device=DEV) if gated else None
    if op == "fc2_bwd":
        s["dy"] = normal((T, H), 1.0 / math.sqrt(H))
        s["y_shared"] = s["act"].float() @ _kn(case, s["ws2"]).float() if gated else None
        s["gate"] = torch.sigmoid(normal((T,), 0.9)) if gated else None
        s["d_h"] = torch.zeros((T, 2 * I_s), dtype=dtype, device=DEV)
        s["d_ws2"] = torch.zeros_like(s["ws2"])
        s["d_gate_logit"] = torch.zeros((T,), device=DEV) if gated else None
    if op == "fc1_bwd":
        s["d_h"] = normal((T, 2 * I_s), 0.02, dtype)
        s["ws1"] = normal(_shape(case, H, 2 * I_s), 0.02, dtype)
        s["d_gate_logit"] = normal((T,), 0.05) if gated else None
        s["d_x"] = torch.zeros((T, H), device=DEV)
        s["d_ws1"] = torch.zeros_like(s["ws1"])
        s["d_w_gate"] = torch.zeros((H,), dtype=dtype, device=DEV) if gated else None
    if own:
        from mixture_experts_ffn_05_amd import binding as B
        s["ws"] = torch.empty((B.moe_shared_train_workspace_bytes(dtype, T, H, I_s),), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def _own_run(s):
    from mixture_experts_ffn_05_amd import binding as B

    case = s["case"]
    op = case["op"]
    if op == "grad_clip":
        B.moe_grad_norm(s["plan"], s["norm"], s["ws"])
        B.moe_grad_clip(s["plan"], s["norm"], case["max_norm"], s["coef"])
        return [s["norm"], s["coef"], *s["flat_outs"]]
    if op == "route_bwd":
        B.moe_route_backward(s["x"], s["w_router"], s["ids"], s["weights"], s["d_weights"], s["d_x"],
                             s["d_w_router"], s["d_bias"], s["ws"], accumulate=True)
        return [s["d_x"], s["d_w_router"], s["d_bias"]]
    layout = B.MOE_W_KN if case["layout"] == "kn" else B.MOE_W_NK
    if op == "fc1_save":
        B.moe_shared_fc1_save(s["x"], s["ws1"], s["act"], s["h_pre"], s["ws"], layout=layout)
        return [s["act"], s["h_pre"]]
    if op == "fc2_save":
        B.moe_shared_fc2_save(s["act"], s["ws2"], s["x"], s["w_gate"], s["y"], s["y_shared"], s["gate"],
                              s["ws"], accumulate=False, layout=layout)
        return [s["y"], s["y_shared"], s["gate"]]
    if op == "fc2_bwd":
        B.moe_shared_fc2_backward(s["dy"], s["act"], s["h_pre"], s["ws2"], s["y_shared"], s["gate"], s["d_h"],
                                  s["d_ws2"], s["d_gate_logit"], s["ws"], layout=layout)
        return [s["d_h"], s["d_ws2"], s["d_gate_logit"]]
    B.moe_shared_fc1_backward(s["d_h"], s["x"], s["ws1"], s["d_gate_logit"], s["w_gate"], s["d_x"], s["d_ws1"],
                              s["d_w_gate"], s["ws"], accumulate=False, layout=layout)
    return [s["d_x"], s["d_ws1"], s["d_w_gate"]]


def run(s):
    if own:
        return _own_run(s)
    case = s["case"]
    op = case["op"]
    if op == "grad_clip":
        # a sum of squares over up to 1e9 elements is long: 64 bits
        norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt()
        coef = (case["max_norm"] / (norm.float() + 1e-6)).clamp(max=1.0)
        [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["outs"])]
        return [norm.float().reshape(1), coef.reshape(1), *s["flat_outs"]]
    dtype = _dtype(case)
    if op == "route_bwd":
        w, dw = s["weights"], s["d_weights"]
        d_sel = w * (dw - (w * dw).sum(1, keepdim=True))
        d_logits = torch.zeros((case["T"], case["E"]), device=DEV).scatter_add_(1, s["ids"].long(), d_sel)
        s["d_x"] += d_logits @ s["w_router"].float().t()
        d_wr = (s["x"].float().t() @ d_logits).to(dtype)
        d_bias = d_logits.sum(0, dtype=torch.float64).float() if case["bias"] else None
        return [s["d_x"], d_wr, d_bias]
    if op == "fc1_save":
        h = s["x"].float() @ _kn(case, s["ws1"]).float()
        g, u = _split(h)
        return [(g / (1 + torch.exp(-g)) * u).to(dtype), h.to(dtype)]
    if op == "fc2_save":
        y = s["act"].float() @ _kn(case, s["ws2"]).float()
        if s["w_gate"] is None:
            return [y, None, None]
        gate = 1 / (1 + torch.exp(-(s["x"].float() * s["w_gate"].float()).sum(1)))
        return [gate[:, None] * y, y, gate]
    if op == "fc2_bwd":
        dy = s["dy"]
        gate = s["gate"]
        d_rows = dy if gate is None else gate[:, None] * dy
        da = d_rows @ _kn(case, s["ws2"]).float().t()
        g, u = _split(s["h_pre"].float())
        sig = 1 / (1 + torch.exp(-g))
        d_h = torch.cat([da * u * sig * (1 + g * (1 - sig)), da * g * sig], dim=1).to(dtype)
        d_w = s["act"].float().t() @ d_rows
        d_w = (d_w if case["layout"] == "kn" else d_w.t()).to(dtype).contiguous()
        d_z = None if gate is None else gate * (1 - gate) * (dy * s["y_shared"]).sum(1)
        return [d_h, d_w, d_z]
    d_h, x = s["d_h"].float(), s["x"].float()
    d_x = d_h @ _kn(case, s["ws1"]).float().t()
    d_w = x.t() @ d_h
    d_w = (d_w if case["layout"] == "kn" else d_w.t()).to(dtype).contiguous()
    if s["w_gate"] is None:
        return [d_x, d_w, None]
    d_x += s["d_gate_logit"][:, None] * s["w_gate"].float()
    return [d_x, d_w, (s["d_gate_logit"][:, None] * x).sum(0).to(dtype)]


def work(case):
    op = case["op"]
    if op == "grad_clip":
        each = [(n, 2 if d == torch.bfloat16 else 4) for n, d in _numels(case, 0)]
        return {"bytes": 2 * sum(n * b for n, b in each), "flops": 3 * sum(n for n, _ in each)}
    e = 2 if case["dt"] == BF16 else 4
    T, H = case["T"], case["H"]
    if op == "route_bwd":
        E, k = case["E"], case["top_k"]
        # x and the router weight in, its gradient out, d_x updated; products with the k selected logits only
        return {"bytes": T * H * e + 2 * H * E * e + 8 * T * H + 12 * T * k + (4 * E if case["bias"] else 0),
                "flops": 4 * T * k * H}
    I_s = case["I_s"]
    gated = case.get("gated", False)
    if op == "fc1_save":
        return {"bytes": e * (T * H + 2 * H * I_s + 3 * T * I_s), "flops": 4 * T * H * I_s}
    if op == "fc2_save":
        return {"bytes": e * (T * I_s + I_s * H) + 4 * T * H + ((e + 4) * T * H + e * H + 4 * T if gated else 0),
                "flops": 2 * T * H * I_s + (2 * T * H if gated else 0)}
    if op == "fc2_bwd":
        return {"bytes": 4 * T * H + e * (5 * T * I_s + 2 * I_s * H) + (4 * T * H + 8 * T if gated else 0),
                "flops": 4 * T * H * I_s + (3 * T * H if gated else 0)}
    return {"bytes": e * (2 * T * I_s + T * H + 4 * H * I_s) + 4 * T * H + (4 * T + 2 * e * H if gated else 0),
            "flops": 8 * T * H * I_s + (4 * T * H if gated else 0)}


def exact(case, seed):
    """The pass's outputs from the formulas, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    D = torch.float64
    if op == "grad_clip":
        sq = torch.zeros((), dtype=D, device=DEV)
        for g in s["grads"]:
            for part in g.split(1 << 26):
                sq += torch.dot(part.to(D), part.to(D))
        norm = torch.sqrt(sq)
        coef = torch.minimum(torch.ones_like(norm), case["max_norm"] / (norm + 1e-6))
        outs = []
        for o in s["flat_outs"]:
            outs.append(torch.cat([g.to(D) for g in s["grads"] if g.dtype == o.dtype]) * coef)
        return [norm.reshape(1), coef.reshape(1), *outs]
    if op == "route_bwd":
        T, E = case["T"], case["E"]
        p, dp = s["weights"].to(D), s["d_weights"].to(D)
        # rows of the softmax's Jacobian: diag(p) - p p^T
        jac = torch.diag_embed(p) - p[:, :, None] * p[:, None, :]
        sel = (jac * dp[:, None, :]).sum(2)
        dense = torch.zeros((T, E), dtype=D, device=DEV)
        for j in range(case["top_k"]):
            rows = torch.arange(T, device=DEV)
            dense[rows, s["ids"][:, j].long()] += sel[:, j]
        return [s["d_x"].to(D) + torch.mm(dense, s["w_router"].to(D).t().contiguous()),
                torch.mm(s["x"].to(D).t().contiguous(), dense), dense.sum(0) if case["bias"] else None]
    nk = case["layout"] == "nk"

    def mat(w):
        w = w.to(D)
        return w.t().contiguous() if nk else w

    def stored(w):
        return w.t().contiguous() if nk else w

    I_s = case["I_s"]
    if op == "fc1_save":
        h = torch.mm(s["x"].to(D), mat(s["ws1"]))
        return [h[:, :I_s] * torch.sigmoid(h[:, :I_s]) * h[:, I_s:], h]
    if op == "fc2_save":
        y = torch.mm(s["act"].to(D), mat(s["ws2"]))
        if not case["gated"]:
            return [y, None, None]
        gate = torch.sigmoid(torch.mv(s["x"].to(D), s["w_gate"].to(D)))
        return [y * gate[:, None], y, gate]
    if op == "fc2_bwd":
        dy = s["dy"].to(D)
        rows = dy * s["gate"].to(D)[:, None] if case["gated"] else dy
        da = torch.mm(rows, mat(s["ws2"]).t().contiguous())
        g, u = s["h_pre"].to(D)[:, :I_s], s["h_pre"].to(D)[:, I_s:]
        sg = torch.sigmoid(g)
        d_h = torch.empty((case["T"], 2 * I_s), dtype=D, device=DEV)
        d_h[:, :I_s] = da * u * (sg + g * sg * (1 - sg))
        d_h[:, I_s:] = da * g * sg
        d_w = stored(torch.mm(s["act"].to(D).t().contiguous(), rows))
        if not case["gated"]:
            return [d_h, d_w, None]
        gate = s["gate"].to(D)
        return [d_h, d_w, (dy * s["y_shared"].to(D)).sum(1) * gate * (1 - gate)]
    d_h, x = s["d_h"].to(D), s["x"].to(D)
    d_x = torch.mm(d_h, mat(s["ws1"]).t().contiguous())
    d_w = stored(torch.mm(x.t().contiguous(), d_h))
    if not case["gated"]:
        return [d_x, d_w, None]
    d_z = s["d_gate_logit"].to(D)
    return [d_x + torch.outer(d_z, s["w_gate"].to(D)), d_w, torch.mv(x.t().contiguous(), d_z)]
