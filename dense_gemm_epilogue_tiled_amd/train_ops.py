"""Training the feed-forward block: the gated linear layer with its backward pass,
the gradients of linear layers, the norms around a block with theirs, and an optimizer's
orthogonalised update.

Raw calls (``gated_linear_bt``, ``linear_backward_raw``, ``gated_linear_backward_raw``,
``sandwich_norm_fwd``, ``sandwich_norm_bwd``, ``orthogonalize_update``) take device pointers
and return the C status; the tensor helpers take GPU tensors with unit column stride
and raise GemmReluError.  Forward and backward passes are calls of their own: nothing is
recorded for autograd, and in grad mode the tensor helpers refuse tensors that
require a gradient.
"""
from __future__ import annotations

import ctypes

from . import GR_FMT_BF16, _ptr, lib
from .mx_ops import _act, _run, _workspace

# Newton-Schulz coefficients, steep at 0 and between 0.7 and 1.2 near 1; published in K. Jordan et al., "Muon: An optimizer
# for hidden layers in neural networks", 2024
QUINTIC = (3.4445, -4.7750, 2.0315)


# ---- raw calls --------------------------------------------------------------------

def _size(call, *args):
    n = ctypes.c_int64(0)
    st = call(*args, ctypes.byref(n))
    return st, int(n.value)


def gated_linear_workspace_size(M, I, H):
    """(status, bytes): the workspace that gated_linear_bt needs (0: none)."""
    return _size(lib().gated_linear_workspace_size, M, I, H)


def gated_linear_bt(M, I, H, X, ldx, W13, ldw, b13, act, C, ldc, GU=None, ldgu=1, fmt=GR_FMT_BF16, workspace=None,
                    workspace_bytes=0, stream=None) -> int:
    """C := act(g) * u, (g, u) = X.W13^T + b13, GU := (g, u) unless None; returns the status code."""
    return lib().gated_linear_bt(M, I, H, _ptr(X), ldx, _ptr(W13), ldw, _ptr(b13), act, _ptr(C), ldc, _ptr(GU), ldgu, fmt,
                                 _ptr(workspace), workspace_bytes, _ptr(stream))


def linear_backward_workspace_size(M, N, K, dY, lddy, X, ldx, W, ldw, dX, lddx, dW, lddw, dB):
    """(status, bytes): the workspace that linear_backward_raw needs with these pointers."""
    return _size(lib().linear_backward_workspace_size, M, N, K, _ptr(dY), lddy, _ptr(X), ldx, _ptr(W), ldw, _ptr(dX), lddx,
                 _ptr(dW), lddw, _ptr(dB))


def linear_backward_raw(M, N, K, dY, lddy, X, ldx, W, ldw, dX, lddx, dW, lddw, dB, fmt=GR_FMT_BF16, workspace=None,
                        workspace_bytes=0, stream=None) -> int:
    """The C call linear_backward: dX := dY.W, dW := dY^T.X, dB := column sums of dY; returns the status code."""
    return lib().linear_backward(M, N, K, _ptr(dY), lddy, _ptr(X), ldx, _ptr(W), ldw, _ptr(dX), lddx, _ptr(dW), lddw,
                                 _ptr(dB), fmt, _ptr(workspace), workspace_bytes, _ptr(stream))


def gated_linear_backward_workspace_size(M, I, H, W13, ldw, dX, lddx, dW13, dB13):
    """(status, bytes): the workspace that gated_linear_backward_raw needs with these pointers."""
    return _size(lib().gated_linear_backward_workspace_size, M, I, H, _ptr(W13), ldw, _ptr(dX), lddx, _ptr(dW13), _ptr(dB13))


def gated_linear_backward_raw(M, I, H, dH, lddh, X, ldx, W13, ldw, GU, ldgu, act, dX, lddx, dW13, lddw, dB13,
                              fmt=GR_FMT_BF16, workspace=None, workspace_bytes=0, stream=None) -> int:
    """The C call gated_linear_backward: dX, dW13, dB13 from dH and what was kept in GU; returns the status code."""
    return lib().gated_linear_backward(M, I, H, _ptr(dH), lddh, _ptr(X), ldx, _ptr(W13), ldw, _ptr(GU), ldgu, act, _ptr(dX),
                                       lddx, _ptr(dW13), lddw, _ptr(dB13), fmt, _ptr(workspace), workspace_bytes,
                                       _ptr(stream))


def sandwich_norm_fwd(M, N, Y, ldy, R, ldr, w, next_w, gate, G, ld_gate, scale, eps, total, ldt, normed, ldn,
                      fmt=GR_FMT_BF16, stream=None) -> int:
    """total := R + scale * gate * norm(Y) * w, normed := norm(total) * next_w; returns the status code."""
    return lib().sandwich_norm_fwd(M, N, _ptr(Y), ldy, _ptr(R), ldr, _ptr(w), _ptr(next_w), _ptr(gate), G, ld_gate, scale,
                                   eps, _ptr(total), ldt, _ptr(normed), ldn, fmt, _ptr(stream))


def sandwich_norm_bwd_workspace_size(M, N, G):
    """(status, bytes): the workspace that sandwich_norm_bwd needs for sums over rows."""
    return _size(lib().sandwich_norm_bwd_workspace_size, M, N, G)


def sandwich_norm_bwd(M, N, dT, ld_dt, dN, ld_dn, Y, ldy, T, ldt, w, next_w, gate, G, ld_gate, scale, eps, dY, ld_dy, dR,
                      ld_dr, dw, dnext_w, dgate, ld_dgate, fmt=GR_FMT_BF16, workspace=None, workspace_bytes=0,
                      stream=None) -> int:
    """The gradients of sandwich_norm_fwd; returns the status code."""
    return lib().sandwich_norm_bwd(M, N, _ptr(dT), ld_dt, _ptr(dN), ld_dn, _ptr(Y), ldy, _ptr(T), ldt, _ptr(w),
                                   _ptr(next_w), _ptr(gate), G, ld_gate, scale, eps, _ptr(dY), ld_dy, _ptr(dR), ld_dr,
                                   _ptr(dw), _ptr(dnext_w), _ptr(dgate), ld_dgate, fmt, _ptr(workspace), workspace_bytes,
                                   _ptr(stream))


def orthogonalize_workspace_size(B, rows, cols):
    """(status, bytes): the workspace that orthogonalize_update needs."""
    return _size(lib().orthogonalize_workspace_size, B, rows, cols)


def orthogonalize_update(B, rows, cols, G, ldg, batch_g, g_fmt, coefficients, steps, scale, eps, out, ldo, batch_o,
                         workspace, workspace_bytes, stream=None) -> int:
    """out := scale * the Newton-Schulz iterate of B matrices G after ``steps``; returns the status code."""
    k = (ctypes.c_float * 3)(*coefficients)
    return lib().orthogonalize_update(B, rows, cols, _ptr(G), ldg, batch_g, g_fmt, k, steps, scale, eps, _ptr(out), ldo,
                                      batch_o, _ptr(workspace), workspace_bytes, _ptr(stream))


# ---- tensors ----------------------------------------------------------------------

def gated_linear(x, w13, b13=None, act="silu", keep=False, out=None, gu_out=None, workspace="auto", stream=None):
    """``(h, gu)``: ``h = act(g) * u`` with ``g, u`` the halves of ``x @ w13.T + b13``.

    ``x`` M x H and ``w13`` 2I x H (the I gate rows, then the I up rows), both float16 or both
    bfloat16; ``b13`` 2I values or None.  g and u are fp32, h is rounded once.  With
    ``keep`` gu is M x 2I, g and u rounded, for gated_linear_backward; else None.
    ``workspace`` as for gemm_relu, but needed where H is not a multiple of 32.
    """
    return _run("gated_linear", "gated_linear_bt", stream, x, w13, b13, _act(act), 1 if keep else 0, out, gu_out,
                _workspace(workspace))


def linear_backward(dy, x, weight, bias=False, input_grad=True, weight_grad=True, dx_out=None, dw_out=None,
                    workspace="auto", stream=None):
    """``(dx, dw, db)``, the gradients of ``y = x @ weight.T + b`` (linear without an activation).

    ``dy`` M x N, ``x`` M x K, ``weight`` N x K, all float16 or all bfloat16.  A gradient that is not asked
    for is None; ``x`` may be None without ``weight_grad``.  Sums over tokens are fp32 in a fixed
    order, rounded once."""
    return _run("linear_backward", "linear_backward", stream, dy, x, weight, 1 if bias else 0, 1 if input_grad else 0,
                1 if weight_grad else 0, dx_out, dw_out, _workspace(workspace))


def gated_linear_backward(dh, x, w13, gu, act="silu", bias=False, input_grad=True, weight_grad=True, dx_out=None,
                          dw_out=None, workspace="auto", stream=None):
    """``(dx, dw13, db13)``, the gradients of gated_linear from ``dh`` (M x I) and the ``gu`` that it
    kept (M x 2I); the other arguments as for gated_linear and linear_backward."""
    return _run("gated_linear_backward", "gated_linear_backward", stream, dh, x, w13, gu, _act(act), 1 if bias else 0,
                1 if input_grad else 0, 1 if weight_grad else 0, dx_out, dw_out, _workspace(workspace))


def sandwich_norm(y, residual, weight=None, next_weight=None, gate=None, scale=1.0, eps=1e-6, next_norm=True,
                  total_out=None, normed_out=None, stream=None):
    """``(total, normed)``: the norm after a block, its gate, the residual and the norm before the next block.

    ``total = residual + scale * gate * norm(y) * weight`` and ``normed = norm(total) * next_weight`` with
    ``norm(v) = v / sqrt(mean(v^2) + eps)`` over the columns, for M x N float16 or bfloat16 tensors (N up to 32768).
    ``gate`` holds N values, or G x N, a row for every M / G consecutive rows.  None stands for
    ones.  With ``next_norm`` false normed is None.  ``total_out`` and ``normed_out`` may be ``y`` or ``residual``.
    """
    return _run("sandwich_norm", "sandwich_norm_fwd", stream, y, residual, weight, next_weight, gate, scale, eps,
                1 if next_norm else 0, total_out, normed_out)


def sandwich_norm_backward(dtotal, dnormed, y, total, weight=None, next_weight=None, gate=None, scale=1.0, eps=1e-6,
                           workspace="auto", stream=None):
    """``(dy, dresidual, dweight, dnext_weight, dgate)`` of sandwich_norm from the gradients of total and normed
    (None for zeros, not both), ``y`` and its ``total``.  The gradient of what is None is None, and without ``dnormed``
    that of next_weight; with no rows those of the weights and gates are zeros."""
    return _run("sandwich_norm_backward", "sandwich_norm_bwd", stream, y, dtotal, dnormed, total, weight, next_weight, gate,
                scale, eps, _workspace(workspace))


def orthogonalize(update, steps=5, coefficients=QUINTIC, scale=1.0, eps=1e-7, out=None, workspace="auto", stream=None):
    """``update`` (rows x cols or batch x rows x cols; float16, bfloat16 or float32) with its singular values
    brought near 1 by ``steps`` Newton-Schulz steps, times ``scale``; bfloat16.

    From ``X = update / (its Frobenius norm + eps)`` each step takes ``X`` to ``a X + (b A + c A A) X``, ``A = X X^T``,
    in fp16 with fp32 sums."""
    a, b, c = coefficients
    return _run("orthogonalize", "orthogonalize_update", stream, update, steps, a, b, c, scale, eps, out,
                _workspace(workspace))
