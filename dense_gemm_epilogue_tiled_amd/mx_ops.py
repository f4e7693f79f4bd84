"""The feed-forward block around the MX products: RMS norm and gated
activation with MX outputs, quantisation, products with MX fp4 weights for few
rows, router and experts.

Raw calls (``rms_norm_mx``, ``gated_act_mx``, ``gemm_w4_bt``, ``moe_route_raw``,
``moe_w4``) take device pointers and return the C status; the tensor helpers
take GPU tensors with unit column stride and raise GemmReluError.  MX fp8 data
is a torch.float8_e4m3fn tensor, MX fp4 data a uint8 tensor of E2M1 pairs (low
nibble first), scales are uint8 E8M0 codes, one per 32 columns.  There are no
gradients: in grad mode the tensor helpers refuse tensors that require one.
"""
from __future__ import annotations

import ctypes

from . import (ACT_CODES, GR_FMT_BF16, GR_FMT_F16, GR_OUT_16, GR_OUT_MXFP4, GR_OUT_MXFP8, GemmReluError, _ptr, lib)

OUT_CODES = {"same": GR_OUT_16, "mxfp8": GR_OUT_MXFP8, "mxfp4": GR_OUT_MXFP4}


# ---- raw calls --------------------------------------------------------------------

def rms_norm_mx(M, N, X, ldx, R, ldr, weight, eps, S, lds, Y, ldy, SY, ld_sy, fmt, out_fmt=GR_OUT_MXFP8,
                stream=None) -> int:
    """Y := RMS norm of the rows of X + R in out_fmt, S := the rounded sum; returns the status code."""
    return lib().rms_norm_mx(M, N, _ptr(X), ldx, _ptr(R), ldr, _ptr(weight), eps, _ptr(S), lds, _ptr(Y), ldy, _ptr(SY),
                             ld_sy, fmt, out_fmt, _ptr(stream))


def gated_act_mx(M, N, G, ldg, U, ldu, act, Y, ldy, SY, ld_sy, fmt, out_fmt=GR_OUT_MXFP8, stream=None) -> int:
    """Y := act(G) * U in out_fmt (U None: act(G)); returns the status code."""
    return lib().gated_act_mx(M, N, _ptr(G), ldg, _ptr(U), ldu, act, _ptr(Y), ldy, _ptr(SY), ld_sy, fmt, out_fmt,
                              _ptr(stream))


def gemm_w4_bt_workspace_size(M, N, K):
    """(status, bytes): the workspace with which gemm_w4_bt is fastest (0: none needed)."""
    n = ctypes.c_int64(0)
    st = lib().gemm_w4_bt_workspace_size(M, N, K, ctypes.byref(n))
    return st, int(n.value)


def gemm_w4_bt(M, N, K, A, lda, Bt, ldbt, scale_b, ld_sb, bias, act, C, ldc, fmt=GR_FMT_BF16, workspace=None,
               workspace_bytes=0, stream=None) -> int:
    """C := act(A.Bt~^T + bias), A, bias and C in fmt, Bt in MX fp4 (N x K); returns the status code."""
    return lib().gemm_w4_bt(M, N, K, _ptr(A), lda, _ptr(Bt), ldbt, _ptr(scale_b), ld_sb, _ptr(bias), act, _ptr(C), ldc,
                            fmt, _ptr(workspace), workspace_bytes, _ptr(stream))


def gemm_mxfp4_linear_bt(M, N, K, A, lda, SA, ld_sa, Bt, ldbt, SB, ld_sb, bias, act, C, ldc, out_fmt=GR_FMT_F16,
                         stream=None) -> int:
    """gemm_mxfp4_bt for any shape (few rows, few tiles, any K % 32 == 0); returns the status code."""
    return lib().gemm_mxfp4_linear_bt(M, N, K, _ptr(A), lda, _ptr(SA), ld_sa, _ptr(Bt), ldbt, _ptr(SB), ld_sb,
                                      _ptr(bias), act, _ptr(C), ldc, out_fmt, _ptr(stream))


def moe_route_workspace_size(T, H, E):
    """(status, bytes): the workspace with which moe_route is fastest (0: none needed)."""
    n = ctypes.c_int64(0)
    st = lib().moe_route_workspace_size(T, H, E, ctypes.byref(n))
    return st, int(n.value)


def moe_route_raw(T, H, E, topk, X, ldx, Wr, ldwr, bias, renorm, ids, weights, fmt=GR_FMT_BF16, workspace=None,
                  workspace_bytes=0, stream=None) -> int:
    """The C call moe_route: top-k experts and softmax weights of T tokens; returns the status code."""
    return lib().moe_route(T, H, E, topk, _ptr(X), ldx, _ptr(Wr), ldwr, _ptr(bias), renorm, _ptr(ids), _ptr(weights),
                           fmt, _ptr(workspace), workspace_bytes, _ptr(stream))


def moe_w4_workspace_size(T, H, I, E, topk):
    """(status, bytes): the workspace that moe_w4 needs."""
    n = ctypes.c_int64(0)
    st = lib().moe_w4_workspace_size(T, H, I, E, topk, ctypes.byref(n))
    return st, int(n.value)


def moe_w4(T, H, I, E, topk, X, ldx, ids, weights, W13, S13, b13, W2, S2, b2, act, C, ldc, fmt, workspace,
           workspace_bytes, stream=None) -> int:
    """The experts of T tokens, MX fp4 weights; returns the status code."""
    return lib().moe_w4(T, H, I, E, topk, _ptr(X), ldx, _ptr(ids), _ptr(weights), _ptr(W13), _ptr(S13), _ptr(b13),
                        _ptr(W2), _ptr(S2), _ptr(b2), act, _ptr(C), ldc, fmt, _ptr(workspace), workspace_bytes,
                        _ptr(stream))


# ---- tensors ----------------------------------------------------------------------
#
# What is done with the tensors themselves (checks, pitches, new outputs and
# scratch) is in csrc/tensors.cpp; here names become codes and streams handles.

_torch = _c = _FMT = _raw_stream = _device = None


def _init():
    global _torch, _c, _FMT, _raw_stream, _device
    import torch
    lib()
    from . import _tensors
    _FMT = {torch.float16: GR_FMT_F16, torch.bfloat16: GR_FMT_BF16}
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch
    _c = _tensors  # last: a set _c means that the others are


def _run(name, status_name, stream, x, *args):
    """Call csrc/tensors.cpp's function `name` on x's device and the given stream (default: the current one), whose
    memory pool new tensors come from."""
    if _c is None:
        _init()
    if not x.is_cuda:
        raise ValueError("%s needs GPU tensors" % name)
    device = x.get_device()
    fn = getattr(_c, name)
    if stream is None and device == _device():
        r = fn(x, *args, _raw_stream(device))
    else:
        with _torch.cuda.device(device):
            if stream is None:
                r = fn(x, *args, _raw_stream(device))
            else:
                if isinstance(stream, int):
                    stream = _torch.cuda.ExternalStream(stream, device=device)
                with _torch.cuda.stream(stream):
                    r = fn(x, *args, stream.cuda_stream)
    if r.__class__ is int:
        raise GemmReluError(r, status_name)
    return r


def _act(act):
    return ACT_CODES[act] if act.__class__ is str else int(act)


def _out(out_format):
    code = OUT_CODES.get(out_format)
    if code is None:
        raise ValueError("out_format must be one of %s" % ", ".join(sorted(OUT_CODES)))
    return code


def _workspace(workspace):
    """True: to be allocated; a tensor or None as given."""
    if workspace.__class__ is str:
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', a tensor or None")
        return True
    return workspace


def rms_norm(x, weight=None, residual=None, eps=1e-6, out_format="mxfp8", out=None, scale_out=None, sum_out=None,
             stream=None):
    """RMS norm of the rows of ``x + residual`` (M x N, float16 or bfloat16).

    Returns ``(y, scale, total)``: y in ``out_format`` ("same" 16 bits, "mxfp8",
    "mxfp4"; the MX formats need N % 32 == 0), its E8M0 scales (None for
    "same") and ``total = x + residual`` rounded to x's type, which is also what is
    normed (None without a residual).  ``sum_out`` may be ``x`` or ``residual``
    itself, and a "same" ``out`` may be ``x`` itself.
    """
    return _run("rms_norm", "rms_norm_mx", stream, x, weight, residual, eps, _out(out_format), out, scale_out, sum_out)


def gated_act(gate, up=None, act="silu", out_format="mxfp8", out=None, scale_out=None, stream=None):
    """``act(gate) * up`` (``up`` None: ``act(gate)``) for M x N float16 or
    bfloat16 tensors; returns ``(y, scale)`` as rms_norm does.  The two halves
    of one M x 2N product are views with its row pitch."""
    return _run("gated_act", "gated_act_mx", stream, gate, up, _act(act), _out(out_format), out, scale_out)


def mx_quantize(x, out_format="mxfp8", out=None, scale_out=None, stream=None):
    """``(elements, scales)`` of the rows of x in "mxfp8" or "mxfp4": operands
    for gemm_mxfp8, gemm_mxfp4 and linear_mxfp4."""
    if out_format == "same":
        raise ValueError("out_format must be mxfp8 or mxfp4")
    return gated_act(x, None, "none", out_format, out, scale_out, stream)


def linear_mxfp4(x, weight, scale, bias=None, act="none", out=None, workspace="auto", stream=None):
    """``act(x @ W.T + bias)`` with 16-bit ``x`` (M x K) and W an N x K MX fp4
    weight (``weight`` N x K/2, ``scale`` N x K/32).  For few rows: the weight
    is read once per 64 rows of x.  ``workspace`` as for gemm_relu."""
    return _run("linear_mxfp4", "gemm_w4_bt", stream, x, weight, scale, bias, _act(act), out, _workspace(workspace))


def gemm_mxfp4(a, scale_a, bt, scale_b, bias=None, act="relu", out_dtype=None, out=None, stream=None, path=None):
    """``out = act(A @ B.T + bias)`` with both operands in MX fp4: ``a`` M x
    K/2 and ``bt`` N x K/2 uint8 (E2M1 pairs), ``scale_a`` M x K/32 and ``scale_b``
    N x K/32 uint8; fp16 or bfloat16 output as for gemm_mxfp8."""
    if _c is None:
        _init()
    kind = out.dtype if out is not None else _torch.float16 if out_dtype is None else out_dtype
    fmt = _FMT.get(kind)
    if fmt is None:
        raise TypeError("the output is float16 or bfloat16")
    return _run("gemm_mxfp4", "gemm_mxfp4_bt", stream, a, scale_a, bt, scale_b, bias, _act(act), fmt, out,
                -1 if path is None else path)


def moe_route(x, router, topk, bias=None, renormalize=True, workspace="auto", stream=None):
    """``(ids, weights)``, T x topk int32 and float32: the topk experts of each
    row of x (T x H) by ``x @ router.T + bias`` (router E x H in x's type, bias E
    float32), in descending order, and the softmax of their logits (over the
    chosen, or over all E with ``renormalize`` false).  ``workspace`` as for
    gemm_relu."""
    return _run("moe_route", "moe_route", stream, x, router, topk, bias, 1 if renormalize else 0,
                _workspace(workspace))


def moe_mxfp4(x, ids, weights, w13, s13, w2, s2, b13=None, b2=None, act="silu", out=None, workspace="auto",
              stream=None):
    """``out[t] = sum_j weights[t, j] * (W2[e] @ h + b2[e])`` with ``h = act(g) *
    u``, ``(g, u) = W13[e] @ x[t] + b13[e]``, ``e = ids[t, j]``.

    ``x`` T x H (float16 or bfloat16), ``ids`` T x topk int32 (an id outside
    [0, E) is passed over), ``weights`` T x topk float32; ``w13`` E x 2I x H/2 and
    ``w2`` E x H x I/2 MX fp4 weights with scales ``s13`` E x 2I x H/32 and ``s2``
    E x H x I/32, all contiguous (an expert's I gate rows, then its I up rows);
    biases ``b13`` E x 2I and ``b2`` E x H in x's type or None.  ``workspace`` as
    for gemm_relu, but needed.
    """
    return _run("moe_mxfp4", "moe_w4", stream, x, ids, weights, w13, s13, w2, s2, b13, b2, _act(act), out,
                _workspace(workspace))
