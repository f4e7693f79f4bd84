"""Plain fp64 forms of the training operators and the bounds of their fp32 computation, for the tests.

Written from the definitions (CPU, float64, no code of the library).  A bound covers what is rounded on the way: fp32
sums (mx_ref.sum_bound, relative to the sum of the products' absolute values), values kept in 16 bits in between, and a
few fp32 steps for each elementary function.  check16 adds half a step of the output.
"""
from __future__ import annotations

import math

import torch

from mx_ref import U32, act, sum_bound

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
QUINTIC = (3.4445, -4.7750, 2.0315)


def make(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * scale).to(TYPES.get(dtype, dtype))


def half(dtype):
    """Half a step of a 16-bit type, relative, and the half step of its subnormal numbers."""
    info = torch.finfo(dtype)
    return info.eps / 2, info.smallest_normal * info.eps / 2


def slope(v, name):
    """The activation's derivative, from the formulas."""
    if name == "relu":
        return (v > 0).double()
    if name == "gelu":
        return 0.5 * torch.special.erfc(-v / math.sqrt(2)) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = torch.sigmoid(2 * c * (v + 0.044715 * v ** 3))
        return s + v * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * v * v)
    if name == "silu":
        s = torch.sigmoid(v)
        return s + v * s * (1 - s)
    if name == "sigmoid":
        return torch.sigmoid(v) * torch.sigmoid(-v)
    if name == "tanh":
        return 1 / torch.cosh(v) ** 2
    return torch.ones_like(v)


# The activations' own error in fp32: 2.5e-7 max(1, |x|) in absolute terms, as the library states for its epilogues, and
# as much again for derivatives; their slopes are at most 1.2.
ACT = 2.5e-7


def gated(x, w13, b13, name):
    """h, gu and the bounds of both before their rounding."""
    xd, wd = x.double(), w13.double()
    gu, mag = xd @ wd.T, xd.abs() @ wd.abs().T
    if b13 is not None:
        gu, mag = gu + b13.double(), mag + b13.double().abs()
    bound = mag * sum_bound(x.shape[1])
    g, u = gu.chunk(2, -1)
    dg, du = bound.chunk(2, -1)
    a = act(g, name)
    da = 1.2 * dg + ACT * (1 + g.abs())
    return a * u, da * (u.abs() + du) + a.abs() * du + 4 * U32 * (a * u).abs(), gu, bound


def products(dy, ddy, x, w):
    """dx, dw, db of y = x w^T and their bounds; ddy: the error that dy comes with."""
    d, m = dy, dy.abs() + ddy
    xd, wd = x.double(), w.double()
    T, N = dy.shape
    out = (d @ wd, d.T @ xd, d.sum(0))
    bound = (m @ wd.abs() * sum_bound(N) + ddy @ wd.abs(), m.T @ xd.abs() * sum_bound(T) + ddy.T @ xd.abs(),
             m.sum(0) * sum_bound(T) + ddy.sum(0))
    return out, bound


def linear_backward(dy, x, w):
    return products(dy.double(), torch.zeros(dy.shape, dtype=torch.float64), x, w)


def gated_backward(dh, x, w13, gu, name):
    """As linear_backward, from the gradients of g and u, which are kept in the operands' type."""
    g, u = gu.double().chunk(2, -1)
    d = dh.double()
    dg, du = d * u * slope(g, name), d * act(g, name)
    err = torch.cat((d.abs() * u.abs() * 2 * ACT * (2 + g.abs()), d.abs() * ACT * (2 + g.abs())), -1)
    dgu = torch.cat((dg, du), -1)
    step, low = half(dh.dtype)
    bound = err + dgu.abs() * (step + 4 * U32) + low
    # a kept value from half a step beyond the type's largest on is an infinity
    info = torch.finfo(dh.dtype)
    over = dgu.abs() >= info.max * (1 + info.eps / 4)
    return products(torch.where(over, torch.copysign(torch.tensor(math.inf, dtype=torch.float64), dgu), dgu), bound, x, w13)


def _norm(v, eps):
    return v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)


def gate_rows(gate, rows):
    """The gate of each row."""
    gate = gate.reshape(-1, gate.shape[-1])
    return gate.repeat_interleave(rows // gate.shape[0], 0)


def sandwich(y, residual, w, next_w, gate, scale, eps):
    """total (before rounding), normed (of the rounded total) and their bounds."""
    M, N = y.shape
    b = _norm(y.double(), eps) * scale
    if w is not None:
        b = b * w.double()
    if gate is not None:
        b = b * gate_rows(gate.double(), M)
    total = residual.double() + b
    # the mean's sum costs at most half its relative bound in the root; 8 more roundings
    rel = (sum_bound(N) / 2 + 8 * U32)
    return total, b.abs() * rel + total.abs() * U32, rel


def next_norm(total, next_w, eps):
    n = _norm(total.double(), eps)
    return n if next_w is None else n * next_w.double()


def sandwich_backward(dt, dn, y, total, w, next_w, gate, scale, eps):
    """(value, bound) of dy, dresidual, dw, dnext_w, dgate."""
    M, N = y.shape
    S = sum_bound(N) + 16 * U32  # of a row's sums and the steps around them
    R = sum_bound(M) + 16 * U32  # of a column's
    yd, z = y.double(), total.double()
    one = torch.ones(N, dtype=torch.float64)
    wd = one if w is None else w.double()
    w2 = one if next_w is None else next_w.double()
    gd = torch.ones(M, N, dtype=torch.float64) if gate is None else gate_rows(gate.double(), M)
    r2 = 1 / torch.sqrt(z.square().mean(-1, keepdim=True) + eps)
    r1 = 1 / torch.sqrt(yd.square().mean(-1, keepdim=True) + eps)
    q, p = z * r2, yd * r1
    d = torch.zeros(M, N, dtype=torch.float64) if dt is None else dt.double()
    err = d.abs() * U32
    dnd = None
    if dn is not None:
        dnd = dn.double()
        dq = dnd * w2
        mean = (dq * q).mean(-1, keepdim=True)
        d = d + r2 * (dq - q * mean)
        err = err + S * r2 * (dq.abs() + q.abs() * (mean.abs() + (dq * q).abs().mean(-1, keepdim=True)))
    dp, ep = d * scale * gd * wd, (err + d.abs() * S) * (scale * gd * wd).abs()
    mean = (dp * p).mean(-1, keepdim=True)
    dy = r1 * (dp - p * mean)
    ey = r1 * (ep + dp.abs() * S + p.abs() * ((ep * p.abs()).mean(-1, keepdim=True)
                                              + S * (mean.abs() + (dp * p).abs().mean(-1, keepdim=True))))
    per = d * scale * p
    eper = (err * scale * p.abs() + per.abs() * (S + R))
    G = 1 if gate is None else gate.reshape(-1, N).shape[0]

    def groups(v):
        return v.reshape(G, -1, N).sum(1)

    out = {"dy": (dy, ey), "dresidual": (d, err), "dw": None, "dnext_w": None, "dgate": None}
    if w is not None:
        out["dw"] = ((per * gd).sum(0), (eper * gd.abs()).sum(0) + (per * gd).abs().sum(0) * (R + G * U32))
    if next_w is not None and dn is not None:
        out["dnext_w"] = ((dnd * q).sum(0), (dnd * q).abs().sum(0) * (S + R))
    if gate is not None:
        out["dgate"] = (groups(per) * wd, (groups(eper) + groups(per.abs()) * R) * wd.abs())
    return out


def newton_schulz(update, steps, coefficients=QUINTIC, eps=1e-7, rounded=False):
    """The iterate, rows x cols or a batch; `rounded`: with operands held in fp16 as the library documents (X times
    2^13, A and B times 2^10), everything else exact."""
    a, b, c = coefficients

    def hold(v, scale):
        return (v * scale).to(torch.float16).double() / scale if rounded else v

    x = update.double()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    x = hold(x / (torch.linalg.matrix_norm(x, keepdim=True) + eps), 2 ** 13)
    unit = torch.eye(x.shape[-2], dtype=torch.float64)
    for s in range(steps):
        m = hold(x @ x.mT, 2 ** 10)
        m = hold(b * m + c * (m @ m) - (b + c) * unit, 2 ** 10)
        x = (a + b + c) * x + m @ x
        if s + 1 < steps:
            x = hold(x, 2 ** 13)
    return x.mT if tall else x
