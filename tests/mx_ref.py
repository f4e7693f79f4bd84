"""Plain fp64 forms of the operators around the MX products, for the tests.

Written from the definitions (CPU, float64, no code of the library).  Weights
are returned with their absolute values' products where an error bound needs
them.
"""
from __future__ import annotations

import math

import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# (emax, lowest exponent of a normal element, fraction bits, largest element)
FORMATS = {"mxfp8": (8, -6, 3, 448.0), "mxfp4": (2, 0, 1, 6.0)}
U32 = 2.0 ** -24  # half a step of fp32, relative


def act(v, name):
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "sigmoid":
        return torch.sigmoid(v)
    if name == "tanh":
        return torch.tanh(v)
    return v


def exponents(y, fmt):
    """Block exponents e of fp64 rows: floor(log2(largest)) - emax in [-127, 127], -127 for zero blocks."""
    amax = y.reshape(y.shape[0], -1, 32).abs().amax(-1)
    e = torch.frexp(amax).exponent - 1 - FORMATS[fmt][0]
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127), amax


def half_step(a, fmt):
    """Half the distance between the elements around a >= 0."""
    _, low, bits, _ = FORMATS[fmt]
    e = (torch.frexp(a).exponent - 1).clamp(min=low)
    return torch.pow(2.0, (e - bits).double()) / 2


def quantise(y, fmt):
    """Elements (fp64 values) and exponents of the MX form of fp64 rows."""
    e, _ = exponents(y, fmt)
    a = y.reshape(y.shape[0], -1, 32) / torch.pow(2.0, e.double())[..., None]
    step = 2 * half_step(a.abs(), fmt)
    most = FORMATS[fmt][3]
    return (torch.round(a / step) * step).clamp(-most, most).reshape(y.shape), e


def unpack4(w):
    """fp64 values of packed E2M1 pairs (low nibble first)."""
    code = torch.stack((w & 15, w >> 4), -1).long().reshape(*w.shape[:-1], -1)
    return E2M1[code & 7] * (1 - 2 * (code >> 3).double())


def weight(w, s):
    """fp64 values of an MX fp4 weight; scale code 255 gives NaN."""
    scale = torch.pow(2.0, s.double() - 127)
    scale = torch.where(s == 255, torch.full_like(scale, float("nan")), scale)
    return unpack4(w) * scale.repeat_interleave(32, -1)


def elements(y, fmt):
    """fp64 element values of an MX output tensor."""
    return unpack4(y) if fmt == "mxfp4" else y.float().double()


def check_mx(y, scale, ref, fmt, delta):
    """Every element of an MX output is a nearest one to the fp64 value, which the fp32 computation may have
    moved by delta, relative; scales likewise."""
    e_got = scale.int() - 127
    e_ref, amax = exponents(ref, fmt)
    low, _ = exponents(ref * (1 - delta), fmt)
    high, _ = exponents(ref * (1 + delta), fmt)
    assert bool(((e_got == e_ref) | (e_got == low) | (e_got == high)).all())
    a = ref.reshape(ref.shape[0], -1, 32) / torch.pow(2.0, e_got.double())[..., None]
    q = elements(y, fmt).reshape(a.shape)
    most = FORMATS[fmt][3]
    held = a.abs().clamp(max=most)
    err = (q - torch.copysign(held, a)).abs()
    assert bool((err <= half_step(held, fmt) + delta * held).all()), float((err - half_step(held, fmt)).max())


def check16(got, ref, dtype, extra):
    """|got - ref| <= half a step of the output type + extra (an absolute bound, elementwise)."""
    info = torch.finfo(dtype)
    got = got.double()
    bound = ref.abs() * (info.eps / 2) + info.smallest_normal * info.eps / 2 + extra
    # values beyond the largest finite one round to infinity
    over = ref.abs() + extra >= info.max * (1 + info.eps / 4)
    bad = ~((got - ref).abs() <= bound) & ~(over & got.isinf())
    assert not bool(bad.any()), "%d of %d off, worst %g over %g" % (
        int(bad.sum()), bad.numel(), float(((got - ref).abs() - bound)[bad].max()), float(bound[bad].max()))


def linear(x, w, s, bias=None, name="none"):
    """act(x W~^T + bias) and the sum of absolute products."""
    wt = weight(w, s)
    v = x.double() @ wt.T
    if bias is not None:
        v = v + bias.double()
    return act(v, name), x.double().abs() @ wt.abs().T + (0 if bias is None else bias.double().abs())


def sum_bound(k):
    """Bound of an fp32 sum of k products, relative to the sum of their absolute values: blocks of 32 inside an MFMA
    (32 roundings at most), one scaled addition per block, a few joins."""
    return (32 + k / 32 + 16) * 2 * U32


def moe(x, ids, weights, w13, s13, w2, s2, b13, b2, name):
    """The layer's output and the bound of an fp32 evaluation of it (h kept to 2^-16)."""
    T, H = x.shape
    E, I = w13.shape[0], w13.shape[1] // 2
    out, bound = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        share = (weights.double() * (ids == e)).sum(1)
        rows = torch.nonzero((ids == e).any(1)).flatten()
        if not len(rows):
            continue
        a, m = weight(w13[e], s13[e]), weight(w2[e], s2[e])
        v, mag = x[rows].double() @ a.T, x[rows].double().abs() @ a.abs().T
        if b13 is not None:
            v, mag = v + b13[e].double(), mag + b13[e].double().abs()
        g, u = v[:, :I], v[:, I:]
        dg, du = mag[:, :I] * sum_bound(H), mag[:, I:] * sum_bound(H)
        ag, p = act(g, name), share[rows][:, None]
        h = ag * u * p
        dh = ((1.2 * dg + 8 * U32 * g.abs()) * u.abs() + ag.abs() * du) * p.abs() + h.abs() * 2.0 ** -16
        out[rows] += h @ m.T
        bound[rows] += dh @ m.abs().T + (h.abs() @ m.abs().T) * (sum_bound(I) + E * U32)
        if b2 is not None:
            out[rows] += p * b2[e].double()
            bound[rows] += (p * b2[e].double()).abs() * 16 * U32
    return out, bound
