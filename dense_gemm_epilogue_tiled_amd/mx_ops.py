"""The feed-forward block around the MX products: RMS norm and gated
activation with MX outputs, quantisation, products with MX fp4 weights for few
rows, router and experts.

Raw calls (``rms_norm_mx``, ``gated_act_mx``, ``gemm_w4_bt``, ``moe_route_raw``,
``moe_w4``) take device pointers and return the C status; the tensor helpers
take GPU tensors with unit column stride and raise GemmReluError.  MX fp8 data
is a torch.float8_e4m3fn tensor, MX fp4 data a uint8 tensor of E2M1 pairs (low
nibble first), scales are uint8 E8M0 codes, one per 32 columns.
"""
from __future__ import annotations

import ctypes

from . import (ACT_CODES, GR_ERR_SCRATCH, GR_FMT_BF16, GR_FMT_F16, GR_OK, GR_OUT_16, GR_OUT_MXFP4, GR_OUT_MXFP8,
               GemmReluError, _ptr, gemm_mxfp4_bt, gemm_mxfp4_bt_forced, lib)

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


def gemm_w4_bt(M, N, K, A, lda, Bt, ldbt, scale_b, ld_sb, bias, act, C, ldc, fmt=GR_FMT_BF16, stream=None) -> int:
    """C := act(A.Bt~^T + bias), A, bias and C in fmt, Bt in MX fp4 (N x K); returns the status code."""
    return lib().gemm_w4_bt(M, N, K, _ptr(A), lda, _ptr(Bt), ldbt, _ptr(scale_b), ld_sb, _ptr(bias), act, _ptr(C), ldc,
                            fmt, _ptr(stream))


def moe_route_raw(T, H, E, topk, X, ldx, Wr, ldwr, bias, renorm, ids, weights, fmt=GR_FMT_BF16, stream=None) -> int:
    """The C call moe_route: top-k experts and softmax weights of T tokens; returns the status code."""
    return lib().moe_route(T, H, E, topk, _ptr(X), ldx, _ptr(Wr), ldwr, _ptr(bias), renorm, _ptr(ids), _ptr(weights),
                           fmt, _ptr(stream))


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

_torch = None


def _t():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _fmt(x):
    torch = _t()
    if x.dtype == torch.bfloat16:
        return GR_FMT_BF16
    if x.dtype == torch.float16:
        return GR_FMT_F16
    raise TypeError("16-bit inputs must be float16 or bfloat16, got %s" % x.dtype)


def _pitch(x, what):
    """Row pitch of a 2-D tensor with unit column stride."""
    rows, cols = x.shape
    stride = x.stride()
    if cols > 1 and rows > 0 and stride[1] != 1:
        raise ValueError("%s needs unit column stride" % what)
    if rows > 1:
        return stride[0] if stride[0] > 0 else 1
    return cols if cols > 0 else 1


def _same(x, other, what):
    """`other` matches x's shape, type and device; its pitch."""
    if other.shape != x.shape or other.dtype != x.dtype:
        raise ValueError("%s must be %s of %s" % (what, tuple(x.shape), x.dtype))
    if other.device != x.device:
        raise ValueError("%s is on another device" % what)
    return _pitch(other, what)


def _vector(x, n, what):
    """The address of a contiguous vector of n values of x's type."""
    if x[0].dtype != x[1].dtype or x[0].dim() != 1 or x[0].shape[0] != n or (n > 1 and x[0].stride(0) != 1):
        raise ValueError("%s must be a contiguous 1-D tensor of %d values of %s" % (what, n, x[1].dtype))
    if x[0].device != x[1].device:
        raise ValueError("%s is on another device" % what)
    return x[0].data_ptr()


def _matrix(x, what):
    if x.dim() != 2:
        raise ValueError("%s must be 2-D" % what)
    if not x.is_cuda:
        raise ValueError("%s must be a GPU tensor" % what)


def _handle(stream, x):
    if stream is None:
        return _t().cuda.current_stream(x.device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _out_code(out_format):
    try:
        return OUT_CODES[out_format]
    except KeyError:
        raise ValueError("out_format must be one of %s" % ", ".join(sorted(OUT_CODES))) from None


def _outputs(x, code, out, scale_out):
    """Output and scale tensors for x's rows in the output format, and their pitches."""
    torch = _t()
    M, N = x.shape
    if code == GR_OUT_16:
        kind, cols = x.dtype, N
        if scale_out is not None:
            raise ValueError("a 16-bit output has no scales")
    else:
        if N % 32:
            raise ValueError("the columns must be a multiple of 32 for an MX output")
        kind, cols = (torch.float8_e4m3fn, N) if code == GR_OUT_MXFP8 else (torch.uint8, N // 2)
    if out is None:
        out = torch.empty((M, cols), dtype=kind, device=x.device)
        ldy = cols if cols > 0 else 1
    else:
        if out.dtype != kind or tuple(out.shape) != (M, cols) or out.device != x.device:
            raise ValueError("out must be %s of %s on the input's device" % ((M, cols), kind))
        ldy = _pitch(out, "out")
    if code == GR_OUT_16:
        return out, ldy, None, 1
    if scale_out is None:
        scale_out = torch.empty((M, N // 32), dtype=torch.uint8, device=x.device)
    elif scale_out.dtype != torch.uint8 or tuple(scale_out.shape) != (M, N // 32) or scale_out.device != x.device:
        raise ValueError("scale_out must be %s of uint8 on the input's device" % ((M, N // 32),))
    return out, ldy, scale_out, _pitch(scale_out, "scale_out")


def rms_norm(x, weight=None, residual=None, eps=1e-6, out_format="mxfp8", out=None, scale_out=None, sum_out=None,
             stream=None):
    """RMS norm of the rows of ``x + residual`` (M x N, float16 or bfloat16).

    Returns ``(y, scale, total)``: y in ``out_format`` ("same" 16 bits, "mxfp8",
    "mxfp4"; the MX formats need N % 32 == 0), its E8M0 scales (None for
    "same") and ``total = x + residual`` rounded to x's type, which is also what is
    normed (None without a residual).  ``sum_out`` may be ``x`` or ``residual``
    itself, and a "same" ``out`` may be ``x`` itself.
    """
    _matrix(x, "x")
    fmt, code = _fmt(x), _out_code(out_format)
    M, N = x.shape
    ldx = _pitch(x, "x")
    w = 0 if weight is None else _vector((weight, x), N, "weight")
    r = s = 0
    ldr = lds = 1
    if residual is not None:
        ldr, r = _same(x, residual, "residual"), residual.data_ptr()
        if sum_out is None:
            sum_out = _t().empty((M, N), dtype=x.dtype, device=x.device)
        lds, s = _same(x, sum_out, "sum_out"), sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    y, ldy, scale, ld_sy = _outputs(x, code, out, scale_out)
    st = lib().rms_norm_mx(M, N, x.data_ptr(), ldx, r, ldr, w, eps, s, lds, y.data_ptr(), ldy,
                           scale.data_ptr() if scale is not None else 0, ld_sy, fmt, code, _handle(stream, x))
    if st != GR_OK:
        raise GemmReluError(st, "rms_norm_mx")
    return y, scale, sum_out


def gated_act(gate, up=None, act="silu", out_format="mxfp8", out=None, scale_out=None, stream=None):
    """``act(gate) * up`` (``up`` None: ``act(gate)``) for M x N float16 or
    bfloat16 tensors; returns ``(y, scale)`` as rms_norm does.  The two halves
    of one M x 2N product are views with its row pitch."""
    _matrix(gate, "gate")
    fmt, code = _fmt(gate), _out_code(out_format)
    M, N = gate.shape
    ldg = _pitch(gate, "gate")
    u, ldu = (0, 1) if up is None else (up.data_ptr(), _same(gate, up, "up"))
    y, ldy, scale, ld_sy = _outputs(gate, code, out, scale_out)
    st = lib().gated_act_mx(M, N, gate.data_ptr(), ldg, u, ldu, ACT_CODES[act] if isinstance(act, str) else int(act),
                            y.data_ptr(), ldy, scale.data_ptr() if scale is not None else 0, ld_sy, fmt, code,
                            _handle(stream, gate))
    if st != GR_OK:
        raise GemmReluError(st, "gated_act_mx")
    return y, scale


def mx_quantize(x, out_format="mxfp8", out=None, scale_out=None, stream=None):
    """``(elements, scales)`` of the rows of x in "mxfp8" or "mxfp4": operands
    for gemm_mxfp8, gemm_mxfp4 and linear_mxfp4."""
    if out_format == "same":
        raise ValueError("out_format must be mxfp8 or mxfp4")
    return gated_act(x, None, "none", out_format, out, scale_out, stream)


def _mxfp4_weight(w, s, k, what):
    """Check an N x K MX fp4 weight and its scales; pitches."""
    torch = _t()
    if w.dtype != torch.uint8 or s.dtype != torch.uint8:
        raise TypeError("%s and its scales must be uint8 (E2M1 pairs, E8M0 codes)" % what)
    if k % 32:
        raise ValueError("K must be a multiple of 32")
    if w.dim() != 2 or w.shape[1] * 2 != k or s.dim() != 2 or tuple(s.shape) != (w.shape[0], k // 32):
        raise ValueError("%s must be N x K/2 with N x K/32 scales for K = %d" % (what, k))
    return _pitch(w, what), _pitch(s, what + "'s scales")


def linear_mxfp4(x, weight, scale, bias=None, act="none", out=None, stream=None):
    """``act(x @ W.T + bias)`` with 16-bit ``x`` (M x K) and W an N x K MX fp4
    weight (``weight`` N x K/2, ``scale`` N x K/32).  For few rows: the weight
    is read once per 64 rows of x."""
    torch = _t()
    _matrix(x, "x")
    fmt = _fmt(x)
    M, K = x.shape
    ldw, ldsw = _mxfp4_weight(weight, scale, K, "weight")
    if weight.device != x.device or scale.device != x.device:
        raise ValueError("weight and scale must be on x's device")
    N = weight.shape[0]
    b = 0 if bias is None else _vector((bias, x), N, "bias")
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
        ldc = N if N > 0 else 1
    else:
        if out.dtype != x.dtype or tuple(out.shape) != (M, N) or out.device != x.device:
            raise ValueError("out must be %s of %s on x's device" % ((M, N), x.dtype))
        ldc = _pitch(out, "out")
    st = lib().gemm_w4_bt(M, N, K, x.data_ptr(), _pitch(x, "x"), weight.data_ptr(), ldw, scale.data_ptr(), ldsw, b,
                          ACT_CODES[act] if isinstance(act, str) else int(act), out.data_ptr(), ldc, fmt,
                          _handle(stream, x))
    if st != GR_OK:
        raise GemmReluError(st, "gemm_w4_bt")
    return out


def gemm_mxfp4(a, scale_a, bt, scale_b, bias=None, act="relu", out_dtype=None, out=None, stream=None, path=None):
    """``out = act(A @ B.T + bias)`` with both operands in MX fp4: ``a`` M x
    K/2 and ``bt`` N x K/2 uint8 (E2M1 pairs), ``scale_a`` M x K/32 and ``scale_b``
    N x K/32 uint8; fp16 or bfloat16 output as for gemm_mxfp8."""
    torch = _t()
    _matrix(a, "a")
    M, K = a.shape[0], a.shape[1] * 2
    lda, ldsa = _mxfp4_weight(a, scale_a, K, "a")
    ldbt, ldsb = _mxfp4_weight(bt, scale_b, K, "bt")
    for t in (scale_a, bt, scale_b):
        if t.device != a.device:
            raise ValueError("operands must be on one device")
    N = bt.shape[0]
    if out is not None:
        out_dtype = out.dtype
    out_dtype = torch.float16 if out_dtype is None else out_dtype
    if out_dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("the output is float16 or bfloat16")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    elif tuple(out.shape) != (M, N) or out.device != a.device:
        raise ValueError("out must be %s on a's device" % ((M, N),))
    bptr = None if bias is None else _vector((bias, out), N, "bias")
    args = (M, N, K, a.data_ptr(), lda, scale_a.data_ptr(), ldsa, bt.data_ptr(), ldbt, scale_b.data_ptr(), ldsb, bptr,
            ACT_CODES[act] if isinstance(act, str) else int(act), out.data_ptr(), _pitch(out, "out"),
            GR_FMT_BF16 if out_dtype == torch.bfloat16 else GR_FMT_F16, _handle(stream, a))
    st = gemm_mxfp4_bt(*args) if path is None else gemm_mxfp4_bt_forced(*args, path)
    if st != GR_OK:
        raise GemmReluError(st, "gemm_mxfp4_bt")
    return out


def moe_route(x, router, topk, bias=None, renormalize=True, stream=None):
    """``(ids, weights)``, T x topk int32 and float32: the topk experts of each
    row of x (T x H) by ``x @ router.T + bias`` (router E x H in x's type, bias E
    float32), in descending order, and the softmax of their logits (over the
    chosen, or over all E with ``renormalize`` false)."""
    torch = _t()
    _matrix(x, "x")
    fmt = _fmt(x)
    T, H = x.shape
    if router.dim() != 2 or router.shape[1] != H or router.dtype != x.dtype or router.device != x.device:
        raise ValueError("router must be E x %d of %s on x's device" % (H, x.dtype))
    E = router.shape[0]
    b = 0
    if bias is not None:
        if bias.dtype != torch.float32 or bias.device != x.device:
            raise ValueError("bias must be float32 on x's device")
        b = _vector((bias, bias), E, "bias")
    k = topk if topk > 0 else 0
    ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
    weights = torch.empty((T, k), dtype=torch.float32, device=x.device)
    st = lib().moe_route(T, H, E, topk, x.data_ptr(), _pitch(x, "x"), router.data_ptr(), _pitch(router, "router"), b,
                         1 if renormalize else 0, ids.data_ptr(), weights.data_ptr(), fmt, _handle(stream, x))
    if st != GR_OK:
        raise GemmReluError(st, "moe_route")
    return ids, weights


def moe_mxfp4(x, ids, weights, w13, s13, w2, s2, b13=None, b2=None, act="silu", out=None, workspace="auto",
              stream=None):
    """``out[t] = sum_j weights[t, j] * (W2[e] @ h + b2[e])`` with ``h = act(g) *
    u``, ``(g, u) = W13[e] @ x[t] + b13[e]``, ``e = ids[t, j]``.

    ``x`` T x H (float16 or bfloat16), ``ids`` T x topk int32 (an id outside
    [0, E) is passed over), ``weights`` T x topk float32; ``w13`` E x 2I x H/2 and
    ``w2`` E x H x I/2 MX fp4 weights with scales ``s13`` E x 2I x H/32 and ``s2``
    E x H x I/32, all contiguous (an expert's I gate rows, then its I up rows);
    biases ``b13`` E x 2I and ``b2`` E x H in x's type or None.  ``workspace`` as
    for gemm_relu.
    """
    torch = _t()
    _matrix(x, "x")
    fmt = _fmt(x)
    T, H = x.shape
    if ids.dtype != torch.int32 or weights.dtype != torch.float32:
        raise TypeError("ids must be int32 and weights float32")
    if ids.dim() != 2 or ids.shape[0] != T or ids.shape != weights.shape:
        raise ValueError("ids and weights must be %d x topk" % T)
    topk = ids.shape[1]
    if w13.dim() != 3 or w13.shape[1] % 2:
        raise ValueError("w13 must be E x 2I x H/2")
    E, I = w13.shape[0], w13.shape[1] // 2
    wanted = ((w13, (E, 2 * I, H // 2)), (s13, (E, 2 * I, H // 32)), (w2, (E, H, I // 2)), (s2, (E, H, I // 32)))
    if H % 32 or I % 32:
        raise ValueError("H and I must be multiples of 32")
    for t, shape in wanted:
        if t.dtype != torch.uint8 or tuple(t.shape) != shape:
            raise ValueError("an expert weight must be uint8 %s, got %s %s" % (shape, t.dtype, tuple(t.shape)))
    for t, shape in ((b13, (E, 2 * I)), (b2, (E, H))):
        if t is not None and (t.dtype != x.dtype or tuple(t.shape) != shape):
            raise ValueError("a bias must be %s of %s" % (shape, x.dtype))
    for t in (ids, weights, w13, s13, w2, s2, b13, b2):
        if t is not None and (not t.is_contiguous() or t.device != x.device):
            raise ValueError("ids, weights, expert weights and biases must be contiguous and on x's device")
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=x.device)
    elif out.dtype != x.dtype or out.shape != x.shape or out.device != x.device:
        raise ValueError("out must be %s of %s on x's device" % (tuple(x.shape), x.dtype))
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto' or a uint8 tensor")
        st, size = moe_w4_workspace_size(T, H, I, E, topk)
        if st != GR_OK:
            raise GemmReluError(st, "moe_w4_workspace_size")
        workspace = torch.empty(size, dtype=torch.uint8, device=x.device)
        if stream is not None and not isinstance(stream, int):
            # the scratch block must not be handed out again before this stream is done with it
            workspace.record_stream(stream)
    elif workspace is None:
        raise GemmReluError(GR_ERR_SCRATCH, "moe_w4")
    st = lib().moe_w4(T, H, I, E, topk, x.data_ptr(), _pitch(x, "x"), ids.data_ptr(), weights.data_ptr(),
                      w13.data_ptr(), s13.data_ptr(), 0 if b13 is None else b13.data_ptr(), w2.data_ptr(),
                      s2.data_ptr(), 0 if b2 is None else b2.data_ptr(),
                      ACT_CODES[act] if isinstance(act, str) else int(act), out.data_ptr(), _pitch(out, "out"), fmt,
                      workspace.data_ptr(), workspace.numel(), _handle(stream, x))
    if st != GR_OK:
        raise GemmReluError(st, "moe_w4")
    return out
