"""Cases and plain forms of the operators of a transformer's feed-forward block on microscaled (OCP MX) data.

Kinds of case:
  norm    RMS norm of x + residual, in 16 bits or as MX fp8 (E4M3 elements, one E8M0 scale per 32 columns)
  gated   act(gate) * up, or x itself, as MX fp8
  quant4  x quantised to MX fp4 and multiplied by an MX fp4 weight
  linear  act(x @ w.T + bias) with 16-bit x and an MX fp4 weight, for few rows
  moe     router, top-k and gated experts with MX fp4 weights, for few tokens

`run` with `own` false computes the operators in fp32 from their formulas; with `own` true it calls the package.
8-bit elements come back as float8_e4m3fn and their scales as float8_e8m0fnu, the values that the bytes stand for.
"""
import math

import torch

own = False

F16 = {"bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


def listed():
    return [
        # one decoded token entering a block whose products take MX fp8
        {"name": "norm_1x4096_bf16_mx8", "op": "norm", "m": 1, "n": 4096, "dtype": "bf16", "out": "mxfp8", "residual": True},
        # a short ragged batch with an odd width, 16-bit output
        {"name": "norm_77x1501_fp16", "op": "norm", "m": 77, "n": 1501, "dtype": "fp16", "out": "same", "residual": True},
        # a long prompt, the widest rows
        {"name": "norm_8192x8192_bf16_mx8", "op": "norm", "m": 8192, "n": 8192, "dtype": "bf16", "out": "mxfp8", "residual": True},
        # a few tokens between the two products of a feed-forward block
        {"name": "gated_8x8192_fp16_silu", "op": "gated", "m": 8, "n": 8192, "dtype": "fp16", "act": "silu", "gate": True},
        # a long prompt between the two products
        {"name": "gated_4100x14336_bf16_silu", "op": "gated", "m": 4100, "n": 14336, "dtype": "bf16", "act": "silu", "gate": True},
        # activations quantised to MX fp4 in front of the product
        {"name": "quant4_512x4096x4096_bf16", "op": "quant4", "m": 512, "n": 4096, "k": 4096, "dtype": "bf16"},
        # one decoded token through a square projection
        {"name": "linear_1x4096x4096_bf16", "op": "linear", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16", "act": "none", "bias": False},
        # an odd number of tokens and of outputs, bias and activation
        {"name": "linear_5x1001x2080_fp16", "op": "linear", "m": 5, "n": 1001, "k": 2080, "dtype": "fp16", "act": "gelu", "bias": True},
        # a decoding batch through the largest projection
        {"name": "linear_16x28672x8192_bf16", "op": "linear", "m": 16, "n": 28672, "k": 8192, "dtype": "bf16", "act": "none", "bias": False},
        # the largest batch that still counts as few rows
        {"name": "linear_64x8192x8192_fp16", "op": "linear", "m": 64, "n": 8192, "k": 8192, "dtype": "fp16", "act": "none", "bias": True},
        # one decoded token through a layer of experts
        {"name": "moe_1_2048x1024_e32k4_bf16", "op": "moe", "m": 1, "h": 2048, "i": 1024, "e": 32, "k": 4, "dtype": "bf16"},
        # a decoding batch that reaches nearly every expert
        {"name": "moe_32_4096x2048_e64k8_bf16", "op": "moe", "m": 32, "h": 4096, "i": 2048, "e": 64, "k": 8, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi, step=1):
    """A whole multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step, max(-(-lo // step), round(v / step))) * step


def draw(rng):
    op = rng.choice(("norm", "gated", "quant4", "linear", "moe"))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "norm":
        out = rng.choice(("mxfp8", "same"))
        n = _spread(rng, 64, 8192, 32 if out == "mxfp8" else 1)
        return {"op": op, "m": _spread(rng, 1, 8192), "n": n, "dtype": dtype, "out": out, "residual": rng.random() < 0.7}
    if op == "gated":
        act = rng.choice(("silu", "gelu_tanh", "none"))
        return {"op": op, "m": _spread(rng, 1, 4100), "n": _spread(rng, 64, 14336, 32), "dtype": dtype, "act": act, "gate": act != "none"}
    if op == "quant4":
        return {"op": op, "m": _spread(rng, 1, 512), "n": _spread(rng, 64, 4096), "k": _spread(rng, 64, 4096, 32), "dtype": dtype}
    if op == "linear":
        m = _spread(rng, 1, 64)
        n = _spread(rng, 64, 28672 if m <= 16 else 8192)
        return {"op": op, "m": m, "n": n, "k": _spread(rng, 64, 8192, 32), "dtype": dtype,
                "act": rng.choice(("none", "silu", "gelu")), "bias": rng.random() < 0.5}
    e = _spread(rng, 4, 64)
    return {"op": op, "m": _spread(rng, 1, 32), "h": _spread(rng, 64, 4096, 32), "i": _spread(rng, 64, 2048, 32),
            "e": e, "k": rng.randint(1, min(8, e)), "dtype": dtype}


def work(case):
    op, m = case["op"], case["m"]
    if op == "norm":
        n = case["n"]
        reads = m * n * 2 * (2 if case["residual"] else 1) + 2 * n
        writes = (2 * m * n if case["residual"] else 0) + (2 * m * n if case["out"] == "same" else m * n + m * n // 32)
        return {"bytes": reads + writes, "flops": 5 * m * n}
    if op == "gated":
        n = case["n"]
        return {"bytes": m * n * (4 if case["gate"] else 2) + m * n + m * n // 32, "flops": 8 * m * n}
    if op in ("quant4", "linear"):
        n, k = case["n"], case["k"]
        return {"bytes": 2 * m * k + n * k // 2 + n * k // 32 + 2 * m * n, "flops": 2 * m * n * k}
    h, i, e, k = case["h"], case["i"], case["e"], case["k"]
    chosen = e * (1 - (1 - k / e) ** m)  # experts that m tokens reach, on average
    weights = chosen * 3 * h * i * (1 / 2 + 1 / 32)
    return {"bytes": weights + 2 * e * h + 4 * m * h + 8 * m * k, "flops": 2 * m * (e * h + k * 3 * h * i)}


def _weight(g, rows, k):
    """An MX fp4 weight: packed E2M1 pairs and E8M0 codes of a layer whose weights are about 0.02."""
    w = torch.randint(0, 256, (*rows, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(118, 122, (*rows, k // 32), generator=g, device="cuda", dtype=torch.uint8)
    return w, s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, op, m = F16[case["dtype"]], case["op"], case["m"]
    st = {"case": case}

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)

    if op == "norm":
        n = case["n"]
        st["x"] = normal(m, n)
        st["residual"] = normal(m, n, scale=3.0) if case["residual"] else None
        st["weight"] = (1 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(t)
    elif op == "gated":
        st["gate"] = normal(m, case["n"], scale=2.0)
        st["up"] = normal(m, case["n"]) if case["gate"] else None
    elif op in ("quant4", "linear"):
        st["x"] = normal(m, case["k"])
        st["w"], st["s"] = _weight(g, (case["n"],), case["k"])
        st["bias"] = normal(case["n"]) if case.get("bias") else None
    else:
        h, i, e = case["h"], case["i"], case["e"]
        st["x"] = normal(m, h)
        st["router"] = normal(e, h, scale=2.0 / math.sqrt(h))
        st["w13"], st["s13"] = _weight(g, (e, 2 * i), h)
        st["w2"], st["s2"] = _weight(g, (e, h), i)
    return st


# ---- the framework's calls --------------------------------------------------------------------------------------

def _run_own(st):
    import dense_gemm_epilogue_tiled_amd as gr
    case = st["case"]
    op = case["op"]
    if op == "norm":
        y, scale, total = gr.rms_norm(st["x"], st["weight"], st["residual"], eps=EPS, out_format=case["out"])
        return _named(y, scale, total)
    if op == "gated":
        y, scale = gr.gated_act(st["gate"], st["up"], act=case["act"], out_format="mxfp8")
        return _named(y, scale, None)
    if op == "quant4":
        q, scale = gr.mx_quantize(st["x"], "mxfp4")
        return gr.gemm_mxfp4(q, scale, st["w"], st["s"], act="none", out_dtype=st["x"].dtype)
    if op == "linear":
        return gr.linear_mxfp4(st["x"], st["w"], st["s"], st["bias"], act=case["act"])
    ids, weights = gr.moe_route(st["x"], st["router"], case["k"])
    out = gr.moe_mxfp4(st["x"], ids, weights, st["w13"], st["s13"], st["w2"], st["s2"], act="silu")
    return {"ids": ids, "weights": weights, "out": out}


def _named(y, scale, total):
    got = {"y": y}
    if scale is not None:
        got["scale"] = scale.view(torch.float8_e8m0fnu)
    if total is not None:
        got["sum"] = total
    return got


# ---- the plain forms, fp32 --------------------------------------------------------------------------------------

def _act(v, name):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v * math.sqrt(0.5))
    return v


def _shared(v, top):
    """Rows of fp32 in blocks of 32, scaled by 2^-e with e = floor(log2(largest)) - top, and the E8M0 codes e + 127."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 1 - top).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    return torch.ldexp(b, -e[..., None]), (e + 127).to(torch.uint8)


def _mx8(v):
    b, code = _shared(v, 8)
    return b.clamp(-448, 448).to(torch.float8_e4m3fn).reshape(v.shape), code


def _mx4(v):
    """The values that v's MX fp4 form stands for: nearest, ties to the even code, at most 6."""
    b, code = _shared(v, 2)
    a = b.abs()
    at = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
          + (a >= 3.5).int() + (a > 5).int())
    q = torch.copysign(torch.tensor(E2M1, device=v.device)[at], b)
    return torch.ldexp(q, code.int()[..., None] - 127).reshape(v.shape)


def _unpacked(w, s):
    """The fp32 values of packed E2M1 pairs (low nibble first) under their E8M0 scales."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=w.device)
    v = torch.stack((lut[(w & 15).int()], lut[(w >> 4).int()]), -1)
    v = v.reshape(*s.shape, 32) * torch.exp2(s.float() - 127)[..., None]
    return v.reshape(*w.shape[:-1], -1)


def _run_plain(st):
    case = st["case"]
    op, t = case["op"], F16[case["dtype"]]
    if op == "norm":
        v, total = st["x"].float(), None
        if st["residual"] is not None:
            total = (v + st["residual"].float()).to(t)
            v = total.float()
        y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * st["weight"].float()
        return _named(y.to(t), None, total) if case["out"] == "same" else _named(*_mx8(y), total)
    if op == "gated":
        v = _act(st["gate"].float(), case["act"])
        return _named(*_mx8(v if st["up"] is None else v * st["up"].float()), None)
    if op == "quant4":
        return (_mx4(st["x"].float()) @ _unpacked(st["w"], st["s"]).T).to(t)
    if op == "linear":
        v = st["x"].float() @ _unpacked(st["w"], st["s"]).T
        return _act(v if st["bias"] is None else v + st["bias"].float(), case["act"]).to(t)
    x = st["x"].float()
    top, ids = (x @ st["router"].float().T).topk(case["k"])
    weights = torch.softmax(top, -1)
    share = torch.zeros(case["e"], x.shape[0], device=x.device).T.scatter_add(1, ids, weights).T
    gate, up = torch.matmul(x, _unpacked(st["w13"], st["s13"]).transpose(1, 2)).chunk(2, -1)
    mid = _act(gate, "silu") * up * share[..., None]
    out = torch.matmul(mid, _unpacked(st["w2"], st["s2"]).transpose(1, 2)).sum(0)
    return {"ids": ids.int(), "weights": weights, "out": out.to(t)}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---- the definitions in fp64 ------------------------------------------------------------------------------------

def _exact_act(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if name == "gelu":
        return v * torch.special.ndtr(v)
    return v


def _exact_mx(v, top, low, bits, most):
    """Values and codes of the MX form of fp64 rows. An element is a multiple of 2^(its exponent - bits), with the
    exponent not below `low`, and not over `most`."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - top, torch.full_like(amax, -127, dtype=torch.int32)).clamp(-127, 127)
    a = b / torch.pow(2.0, e.double())
    step = torch.pow(2.0, (torch.frexp(a)[1] - 1).clamp(min=low).double() - bits)
    q = (torch.round(a / step) * step).clamp(-most, most)
    return q, e


def _exact_weight(w, s):
    sign = 1.0 - 2.0 * torch.stack(((w >> 3) & 1, w >> 7), -1).double()
    code = torch.stack((w & 7, (w >> 4) & 7), -1)
    high, low = (code >> 1).double(), (code & 1).double()
    v = sign * torch.where(high > 0, torch.pow(2.0, high - 1) * (1 + low / 2), low / 2)
    return (v.flatten(-2).unflatten(-1, (-1, 32)) * torch.pow(2.0, s.double() - 127).unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    op, t = case["op"], F16[case["dtype"]]
    if op in ("norm", "gated"):
        total = None
        if op == "norm":
            v = st["x"].double()
            if st["residual"] is not None:
                total = v + st["residual"].double()
                v = total.to(t).double()
            v = v / torch.sqrt(v.square().sum(-1, keepdim=True) / case["n"] + EPS) * st["weight"].double()
            if case["out"] == "same":
                return _named(v, None, total)
        else:
            v = _exact_act(st["gate"].double(), case["act"])
            if st["up"] is not None:
                v = v * st["up"].double()
        q, e = _exact_mx(v, 8, -6, 3, 448.0)
        return _named(q.flatten(-2).to(torch.float8_e4m3fn), (e + 127).squeeze(-1).to(torch.uint8), total)
    if op == "quant4":
        q, e = _exact_mx(st["x"].double(), 2, 0, 1, 6.0)
        return (q * torch.pow(2.0, e.double())).flatten(-2) @ _exact_weight(st["w"], st["s"]).T
    if op == "linear":
        v = st["x"].double() @ _exact_weight(st["w"], st["s"]).T
        return _exact_act(v if st["bias"] is None else v + st["bias"].double(), case["act"])
    x = st["x"].double()
    logits = x @ st["router"].double().T
    order = torch.argsort(logits, dim=-1, descending=True, stable=True)[:, : case["k"]]
    chosen = torch.exp(logits.gather(1, order) - logits.amax(-1, keepdim=True))
    weights = chosen / chosen.sum(-1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(case["e"]):
        row, slot = torch.nonzero(order == e, as_tuple=True)
        if row.numel():
            gate, up = (x[row] @ _exact_weight(st["w13"][e], st["s13"][e]).T).split(case["i"], -1)
            y = (_exact_act(gate, "silu") * up) @ _exact_weight(st["w2"][e], st["s2"][e]).T
            out[row] += y * weights[row, slot].unsqueeze(-1)
    return {"ids": order.int(), "weights": weights, "out": out}
