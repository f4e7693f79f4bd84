"""Cases and plain forms of the operators that train a transformer's feed-forward block.

Kinds of case:
  gated       h = act(x Wg^T) * (x Wu^T), both projections in one product, with or without what the backward pass needs
  gated_bwd   its gradients: dx and those of the stacked weight, from dh and the kept products
  linear_bwd  the gradients of y = x W^T + b
  norm        total = residual + scale * gate * norm(y) * w, and the next block's norm(total) * w_next
  norm_bwd    its gradients, those of the weights and of the gates among them
  ortho       an update made orthogonal by Newton-Schulz products

`run` with `own` false computes the operators in fp32 from their formulas; with `own` true it calls the package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
SCALE = 0.5  # of a block's output on its way into the residual
STEPS = 5
QUINTIC = (3.4445, -4.7750, 2.0315)


def listed():
    return [
        # one decoded token
        {"name": "gated_1x4096x14336_bf16", "op": "gated", "m": 1, "h": 4096, "i": 14336, "dtype": "bf16", "act": "silu", "keep": False},
        # a short batch with an odd width, on the way to a backward pass
        {"name": "gated_77x2080x1501_fp16", "op": "gated", "m": 77, "h": 2080, "i": 1501, "dtype": "fp16", "act": "gelu_tanh", "keep": True},
        # a training batch through the widest projection
        {"name": "gated_8192x4096x14336_bf16", "op": "gated", "m": 8192, "h": 4096, "i": 14336, "dtype": "bf16", "act": "silu", "keep": True},
        # its way back
        {"name": "gated_bwd_8192x4096x14336_bf16", "op": "gated_bwd", "m": 8192, "h": 4096, "i": 14336, "dtype": "bf16", "act": "silu"},
        # a projection out of the block, a ragged batch of a small model, with a bias
        {"name": "linear_bwd_333x1001x2080_fp16", "op": "linear_bwd", "m": 333, "n": 1001, "k": 2080, "dtype": "fp16", "bias": True},
        # a training batch through the projection out of the block
        {"name": "linear_bwd_8192x4096x8192_bf16", "op": "linear_bwd", "m": 8192, "n": 4096, "k": 8192, "dtype": "bf16", "bias": False},
        # one decoded token between two blocks
        {"name": "norm_1x4096_bf16", "op": "norm", "m": 1, "n": 4096, "dtype": "bf16", "gates": 1},
        # a training batch of the widest rows, a gate for each of its sequences
        {"name": "norm_8192x8192_bf16", "op": "norm", "m": 8192, "n": 8192, "dtype": "bf16", "gates": 4},
        # its way back
        {"name": "norm_bwd_8192x8192_bf16", "op": "norm_bwd", "m": 8192, "n": 8192, "dtype": "bf16", "gates": 4},
        # small matrices of one shape together
        {"name": "ortho_8x256x1024_bf16", "op": "ortho", "batch": 8, "rows": 256, "cols": 1024, "dtype": "bf16"},
        # one odd matrix, taller than wide
        {"name": "ortho_1501x1000_fp32", "op": "ortho", "batch": 1, "rows": 1501, "cols": 1000, "dtype": "fp32"},
        # a wide projection's momentum in fp32
        {"name": "ortho_4096x8192_fp32", "op": "ortho", "batch": 1, "rows": 4096, "cols": 8192, "dtype": "fp32"},
    ]


def _spread(rng, lo, hi, step=1):
    """A whole multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step, max(-(-lo // step), round(v / step))) * step


def _width(rng, lo, hi):
    """Three widths in four are whole multiples of 32, as most layers' are."""
    return _spread(rng, lo, hi, 32 if rng.random() < 0.75 else 1)


def draw(rng):
    op = rng.choice(("gated", "gated_bwd", "linear_bwd", "norm", "norm_bwd", "ortho"))
    dtype = rng.choice(("bf16", "fp16"))
    if op in ("gated", "gated_bwd"):
        case = {"op": op, "m": _spread(rng, 1, 8192), "h": _width(rng, 64, 4096), "i": _width(rng, 64, 14336), "dtype": dtype,
                "act": rng.choice(("silu", "gelu", "gelu_tanh", "relu"))}
        if op == "gated":
            case["keep"] = rng.random() < 0.5
        return case
    if op == "linear_bwd":
        return {"op": op, "m": _spread(rng, 1, 8192), "n": _width(rng, 64, 4096), "k": _width(rng, 64, 8192), "dtype": dtype,
                "bias": rng.random() < 0.5}
    if op in ("norm", "norm_bwd"):
        gates = rng.choice((0, 1, 4))
        m = _spread(rng, max(1, gates), 8192, max(1, gates))
        return {"op": op, "m": m, "n": _width(rng, 64, 8192), "dtype": dtype, "gates": gates}
    rows, cols = _width(rng, 16, 4096), _width(rng, 16, 4096)
    batch = _spread(rng, 1, 8) if rows * cols <= 1 << 20 else 1
    return {"op": op, "batch": batch, "rows": rows, "cols": cols, "dtype": rng.choice(("bf16", "fp16", "fp32"))}


def work(case):
    op = case["op"]
    if op in ("gated", "gated_bwd"):
        m, h, i = case["m"], case["h"], case["i"]
        weight = 4 * h * i
        if op == "gated":
            return {"bytes": 2 * m * h + weight + 2 * m * i * (3 if case["keep"] else 1), "flops": 4 * m * h * i}
        return {"bytes": 4 * m * h + 2 * weight + 6 * m * i, "flops": 8 * m * h * i}
    if op == "linear_bwd":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * (m * n + 2 * m * k + 2 * n * k + (n if case["bias"] else 0)), "flops": 4 * m * n * k}
    if op in ("norm", "norm_bwd"):
        m, n = case["m"], case["n"]
        params = 2 * n * (2 + case["gates"])
        if op == "norm":
            return {"bytes": 8 * m * n + params, "flops": 10 * m * n}
        return {"bytes": 12 * m * n + 2 * params, "flops": 30 * m * n}
    r, c = sorted((case["rows"], case["cols"]))
    size = 4 if case["dtype"] == "fp32" else 2
    # the two symmetric products cost half
    return {"bytes": case["batch"] * r * c * (size + 2), "flops": case["batch"] * STEPS * (r * r * c + r ** 3 + 2 * r * r * c)}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, op = TYPES[case["dtype"]], case["op"]
    st = {"case": case}

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)

    if op in ("gated", "gated_bwd"):
        m, h, i = case["m"], case["h"], case["i"]
        st["x"] = normal(m, h)
        st["w13"] = normal(2 * i, h, scale=1.5 / math.sqrt(h))
        if op == "gated_bwd":
            st["gu"] = (st["x"].float() @ st["w13"].float().T).to(t)
            st["dh"] = normal(m, i, scale=0.1)
    elif op == "linear_bwd":
        m, n, k = case["m"], case["n"], case["k"]
        st["x"] = normal(m, k)
        st["w"] = normal(n, k, scale=1 / math.sqrt(k))
        st["dy"] = normal(m, n, scale=0.1)
    elif op in ("norm", "norm_bwd"):
        m, n, gates = case["m"], case["n"], case["gates"]
        st["y"] = normal(m, n, scale=0.7)
        st["w"] = (1 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(t)
        st["next_w"] = (1 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(t)
        st["gate"] = normal(gates, n) if gates else None
        if op == "norm":
            st["residual"] = normal(m, n, scale=2.0)
        else:
            st["total"] = normal(m, n, scale=2.0)
            st["dtotal"], st["dnormed"] = normal(m, n, scale=0.1), normal(m, n, scale=0.1)
    else:
        b, r, c = case["batch"], case["rows"], case["cols"]
        # a gradient's momentum: a few strong directions over a broad rest
        k = max(1, min(r, c) // 64)
        strong = torch.randn(b, r, k, generator=g, device="cuda") @ torch.randn(b, k, c, generator=g, device="cuda")
        v = torch.randn(b, r, c, generator=g, device="cuda") + strong / math.sqrt(k)
        st["update"] = (v * 1e-2).to(t)[0] if b == 1 else (v * 1e-2).to(t)
    return st


# ---- the framework's calls --------------------------------------------------------------------------------------

def _run_own(st):
    import dense_gemm_epilogue_tiled_amd as gr
    case = st["case"]
    op = case["op"]
    if op == "gated":
        h, gu = gr.gated_linear(st["x"], st["w13"], act=case["act"], keep=case["keep"])
        return {"h": h, "gu": gu}
    if op == "gated_bwd":
        dx, dw, _ = gr.gated_linear_backward(st["dh"], st["x"], st["w13"], st["gu"], act=case["act"])
        return {"dx": dx, "dw13": dw}
    if op == "linear_bwd":
        dx, dw, db = gr.linear_backward(st["dy"], st["x"], st["w"], bias=case["bias"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "norm":
        total, normed = gr.sandwich_norm(st["y"], st["residual"], st["w"], st["next_w"], st["gate"], scale=SCALE, eps=EPS)
        return {"total": total, "normed": normed}
    if op == "norm_bwd":
        dy, dres, dw, dnext, dgate = gr.sandwich_norm_backward(st["dtotal"], st["dnormed"], st["y"], st["total"], st["w"],
                                                               st["next_w"], st["gate"], scale=SCALE, eps=EPS)
        return {"dy": dy, "dresidual": dres, "dw": dw, "dnext_w": dnext, "dgate": dgate}
    return gr.orthogonalize(st["update"], steps=STEPS, coefficients=QUINTIC)


# ---- the plain forms, fp32 --------------------------------------------------------------------------------------

def _act(v, name):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v * math.sqrt(0.5))
    if name == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return torch.where(v > 0, v, torch.zeros_like(v))


def _slope(v, name):
    """The activation's derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    if name == "gelu":
        return 0.5 * torch.special.erfc(-v * math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-2 * c * (v + 0.044715 * v * v * v)))
        return s + v * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * v * v)
    return (v > 0).float()


def _gates(st):
    """The gate of each row, or 1."""
    if st["gate"] is None:
        return 1.0
    return st["gate"].float().repeat_interleave(st["y"].shape[0] // st["gate"].shape[0], 0)


def _run_plain(st):
    case = st["case"]
    op, t = case["op"], TYPES[case["dtype"]]
    if op == "gated":
        gu = st["x"].float() @ st["w13"].float().T
        g, u = gu.chunk(2, -1)
        return {"h": (_act(g, case["act"]) * u).to(t), "gu": gu.to(t) if case["keep"] else None}
    if op == "gated_bwd":
        g, u = st["gu"].float().chunk(2, -1)
        dh = st["dh"].float()
        dgu = torch.cat((dh * u * _slope(g, case["act"]), dh * _act(g, case["act"])), -1)
        return {"dx": (dgu @ st["w13"].float()).to(t), "dw13": (dgu.T @ st["x"].float()).to(t)}
    if op == "linear_bwd":
        dy = st["dy"].float()
        return {"dx": (dy @ st["w"].float()).to(t), "dw": (dy.T @ st["x"].float()).to(t),
                "db": dy.sum(0).to(t) if case["bias"] else None}
    if op == "norm":
        y = st["y"].float()
        p = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        total = (st["residual"].float() + SCALE * _gates(st) * (p * st["w"].float())).to(t)
        v = total.float()
        return {"total": total, "normed": (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * st["next_w"].float()).to(t)}
    if op == "norm_bwd":
        v, dn = st["total"].float(), st["dnormed"].float()
        r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
        q, dq = v * r, dn * st["next_w"].float()
        d = st["dtotal"].float() + r * (dq - q * (dq * q).mean(-1, keepdim=True))
        y, w, gate = st["y"].float(), st["w"].float(), _gates(st)
        r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        p = y * r
        db = d * SCALE * gate
        dp = db * w
        dgate = None
        if st["gate"] is not None:
            dgate = (d * SCALE * (p * w)).reshape(case["gates"], -1, case["n"]).sum(1).to(t)
        return {"dy": (r * (dp - p * (dp * p).mean(-1, keepdim=True))).to(t), "dresidual": d.to(t), "dw": (db * p).sum(0).to(t),
                "dnext_w": (dn * q).sum(0).to(t), "dgate": dgate}
    x = st["update"].float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-2, -1)
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + 1e-7)
    a, b, c = QUINTIC
    for _ in range(STEPS):
        s = x @ x.transpose(-2, -1)
        x = a * x + (b * s + c * (s @ s)) @ x
    return (x.transpose(-2, -1) if tall else x).to(torch.bfloat16)


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---- the definitions in fp64 ------------------------------------------------------------------------------------

def _exact_act(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        return v * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v.clamp(min=0)


def _exact_norm(v, w):
    return v / torch.sqrt(v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS) * w


def _exact_branch(y, w, gate):
    out = _exact_norm(y, w) * SCALE
    return out if gate is None else (out.unflatten(0, (gate.shape[0], -1)) * gate[:, None]).flatten(0, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op, t = case["op"], TYPES[case["dtype"]]
    v = {k: x.double() for k, x in st.items() if isinstance(x, torch.Tensor)}
    if op == "gated":
        i = case["i"]
        gate, up = torch.mm(v["x"], v["w13"][:i].t()), torch.mm(v["x"], v["w13"][i:].t())
        return {"h": _exact_act(gate, case["act"]) * up, "gu": torch.cat((gate, up), 1) if case["keep"] else None}
    if op == "gated_bwd":
        with torch.enable_grad():
            gu = v["gu"].requires_grad_()
            h = _exact_act(gu[:, : case["i"]], case["act"]) * gu[:, case["i"]:]
            dgu, = torch.autograd.grad(h, gu, v["dh"])
        return {"dx": torch.mm(dgu, v["w13"]), "dw13": torch.mm(dgu.t(), v["x"])}
    if op == "linear_bwd":
        return {"dx": torch.mm(v["dy"], v["w"]), "dw": torch.mm(v["dy"].t(), v["x"]),
                "db": v["dy"].sum(0) if case["bias"] else None}
    if op == "norm":
        total = v["residual"] + _exact_branch(v["y"], v["w"], v.get("gate"))
        return {"total": total, "normed": _exact_norm(total.to(t).double(), v["next_w"])}
    if op == "norm_bwd":
        with torch.enable_grad():
            total, next_w = v["total"].requires_grad_(), v["next_w"].requires_grad_()
            d, dnext = torch.autograd.grad(_exact_norm(total, next_w), (total, next_w), v["dnormed"])
            d = d + v["dtotal"]
            leaves = [v["y"].requires_grad_(), v["w"].requires_grad_()]
            if "gate" in v:
                leaves.append(v["gate"].requires_grad_())
            got = torch.autograd.grad(_exact_branch(v["y"], v["w"], v.get("gate")), leaves, d)
        return {"dy": got[0], "dresidual": d, "dw": got[1], "dnext_w": dnext, "dgate": got[2] if len(got) > 2 else None}
    x = v["update"]
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + 1e-7)
    a, b, c = QUINTIC
    for _ in range(STEPS):  # the polynomial from the narrow side: the same matrix either way
        if x.shape[-2] <= x.shape[-1]:
            s = torch.matmul(x, x.mT)
            x = a * x + torch.matmul(s, b * x + c * torch.matmul(s, x))
        else:
            s = torch.matmul(x.mT, x)
            x = a * x + torch.matmul(b * x + c * torch.matmul(x, s), s)
    return x
