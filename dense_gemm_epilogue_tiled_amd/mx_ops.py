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
               GemmReluError, _ptr, gemm_mxfp4_bt_forced, lib)

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
# A decoding step calls these for microseconds of GPU work, so what they do on
# the host counts: types are looked up in dictionaries, the current stream is read as a
# raw handle, and tensors are asked once for what is needed of them.

_torch = _l = _FMT = _OUT_TYPE = _raw_stream = _device = None


def _init():
    global _torch, _l, _FMT, _OUT_TYPE, _raw_stream, _device
    import torch
    _l = lib()
    _FMT = {torch.float16: GR_FMT_F16, torch.bfloat16: GR_FMT_BF16}
    _OUT_TYPE = {GR_OUT_MXFP8: torch.float8_e4m3fn, GR_OUT_MXFP4: torch.uint8}
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _device = torch.cuda.current_device
    _torch = torch


def _matrix(x, what):
    """x's format code, rows, columns and pitch; x is a 2-D 16-bit GPU tensor with unit column stride."""
    if _torch is None:
        _init()
    fmt = _FMT.get(x.dtype)
    if fmt is None:
        raise TypeError("%s must be float16 or bfloat16, got %s" % (what, x.dtype))
    if x.dim() != 2:
        raise ValueError("%s must be 2-D" % what)
    if not x.is_cuda:
        raise ValueError("%s must be a GPU tensor" % what)
    rows, cols = x.shape
    return fmt, rows, cols, _pitch(x, rows, cols, what)


def _pitch(x, rows, cols, what):
    """Row pitch of a 2-D tensor with unit column stride."""
    row, col = x.stride()
    if col != 1 and cols > 1 and rows > 0:
        raise ValueError("%s needs unit column stride" % what)
    if rows > 1:
        return row if row > 0 else 1
    return cols if cols > 0 else 1


def _like(x, other, rows, cols, kind, what):
    """The pitch of `other`, which is rows x cols of type `kind` on x's device."""
    if other.dtype != kind or other.shape != (rows, cols):
        raise ValueError("%s must be %s of %s" % (what, (rows, cols), kind))
    if other.get_device() != x.get_device():
        raise ValueError("%s is on another device" % what)
    return _pitch(other, rows, cols, what)


def _vector(v, x, n, kind, what):
    """The address of a contiguous vector of n values of type `kind` on x's device."""
    if v.dtype != kind or v.shape != (n,) or (n > 1 and v.stride(0) != 1):
        raise ValueError("%s must be a contiguous 1-D tensor of %d values of %s" % (what, n, kind))
    if v.get_device() != x.get_device():
        raise ValueError("%s is on another device" % what)
    return v.data_ptr()


def _empty(x, shape, kind, stream):
    """A new tensor next to x, of the stream that will use it."""
    if stream is None:
        return x.new_empty(shape, dtype=kind)
    if isinstance(stream, int):
        stream = _torch.cuda.ExternalStream(stream, device=x.device)
    with _torch.cuda.stream(stream):
        return x.new_empty(shape, dtype=kind)


def _act(act):
    return ACT_CODES[act] if act.__class__ is str else int(act)


def _run(fn, x, args, stream, what):
    """Call the library on x's device and the given stream (default: the current one)."""
    device = x.get_device()
    if stream is None:
        handle = _raw_stream(device)
    else:
        handle = stream if isinstance(stream, int) else stream.cuda_stream
    if device == _device():
        st = fn(*args, handle)
    else:
        with _torch.cuda.device(device):
            st = fn(*args, handle)
    if st != GR_OK:
        raise GemmReluError(st, what)


def _outputs(x, M, N, out_format, out, scale_out, stream):
    """The output code, the output and its pitch, the scales and theirs."""
    code = OUT_CODES.get(out_format)
    if code is None:
        raise ValueError("out_format must be one of %s" % ", ".join(sorted(OUT_CODES)))
    if code == GR_OUT_16:
        if scale_out is not None:
            raise ValueError("a 16-bit output has no scales")
        kind, cols = x.dtype, N
    else:
        if N % 32:
            raise ValueError("the columns must be a multiple of 32 for an MX output")
        kind, cols = _OUT_TYPE[code], N if code == GR_OUT_MXFP8 else N // 2
    if out is None:
        out, ldy = _empty(x, (M, cols), kind, stream), cols if cols > 0 else 1
    else:
        ldy = _like(x, out, M, cols, kind, "out")
    if code == GR_OUT_16:
        return code, out, ldy, None, 1
    blocks = N // 32
    if scale_out is None:
        return code, out, ldy, _empty(x, (M, blocks), _torch.uint8, stream), blocks if blocks > 0 else 1
    return code, out, ldy, scale_out, _like(x, scale_out, M, blocks, _torch.uint8, "scale_out")


def rms_norm(x, weight=None, residual=None, eps=1e-6, out_format="mxfp8", out=None, scale_out=None, sum_out=None,
             stream=None):
    """RMS norm of the rows of ``x + residual`` (M x N, float16 or bfloat16).

    Returns ``(y, scale, total)``: y in ``out_format`` ("same" 16 bits, "mxfp8",
    "mxfp4"; the MX formats need N % 32 == 0), its E8M0 scales (None for
    "same") and ``total = x + residual`` rounded to x's type, which is also what is
    normed (None without a residual).  ``sum_out`` may be ``x`` or ``residual``
    itself, and a "same" ``out`` may be ``x`` itself.
    """
    fmt, M, N, ldx = _matrix(x, "x")
    w = 0 if weight is None else _vector(weight, x, N, x.dtype, "weight")
    r = s = 0
    ldr = lds = 1
    if residual is not None:
        ldr, r = _like(x, residual, M, N, x.dtype, "residual"), residual.data_ptr()
        if sum_out is None:
            sum_out, lds = _empty(x, (M, N), x.dtype, stream), N if N > 0 else 1
        else:
            lds = _like(x, sum_out, M, N, x.dtype, "sum_out")
        s = sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    code, y, ldy, scale, ld_sy = _outputs(x, M, N, out_format, out, scale_out, stream)
    _run(_l.rms_norm_mx, x, (M, N, x.data_ptr(), ldx, r, ldr, w, eps, s, lds, y.data_ptr(), ldy,
                             0 if scale is None else scale.data_ptr(), ld_sy, fmt, code), stream, "rms_norm_mx")
    return y, scale, sum_out


def gated_act(gate, up=None, act="silu", out_format="mxfp8", out=None, scale_out=None, stream=None):
    """``act(gate) * up`` (``up`` None: ``act(gate)``) for M x N float16 or
    bfloat16 tensors; returns ``(y, scale)`` as rms_norm does.  The two halves
    of one M x 2N product are views with its row pitch."""
    fmt, M, N, ldg = _matrix(gate, "gate")
    u, ldu = (0, 1) if up is None else (up.data_ptr(), _like(gate, up, M, N, gate.dtype, "up"))
    code, y, ldy, scale, ld_sy = _outputs(gate, M, N, out_format, out, scale_out, stream)
    _run(_l.gated_act_mx, gate, (M, N, gate.data_ptr(), ldg, u, ldu, _act(act), y.data_ptr(), ldy,
                                 0 if scale is None else scale.data_ptr(), ld_sy, fmt, code), stream, "gated_act_mx")
    return y, scale


def mx_quantize(x, out_format="mxfp8", out=None, scale_out=None, stream=None):
    """``(elements, scales)`` of the rows of x in "mxfp8" or "mxfp4": operands
    for gemm_mxfp8, gemm_mxfp4 and linear_mxfp4."""
    if out_format == "same":
        raise ValueError("out_format must be mxfp8 or mxfp4")
    return gated_act(x, None, "none", out_format, out, scale_out, stream)


def _mxfp4_weight(w, s, x, k, what):
    """The rows of an N x K MX fp4 weight on x's device, its pitch and its scales'."""
    if w.dtype != _torch.uint8 or s.dtype != _torch.uint8:
        raise TypeError("%s and its scales must be uint8 (E2M1 pairs, E8M0 codes)" % what)
    if k % 32:
        raise ValueError("K must be a multiple of 32")
    if w.dim() != 2 or w.shape[1] * 2 != k or s.shape != (w.shape[0], k // 32):
        raise ValueError("%s must be N x K/2 with N x K/32 scales for K = %d" % (what, k))
    if w.get_device() != x.get_device() or s.get_device() != x.get_device():
        raise ValueError("%s and its scales must be on one device with the other operands" % what)
    n = w.shape[0]
    return n, _pitch(w, n, k // 2, what), _pitch(s, n, k // 32, what + "'s scales")


def linear_mxfp4(x, weight, scale, bias=None, act="none", out=None, workspace="auto", stream=None):
    """``act(x @ W.T + bias)`` with 16-bit ``x`` (M x K) and W an N x K MX fp4
    weight (``weight`` N x K/2, ``scale`` N x K/32).  For few rows: the weight
    is read once per 64 rows of x.  ``workspace`` as for gemm_relu."""
    fmt, M, K, ldx = _matrix(x, "x")
    N, ldw, ldsw = _mxfp4_weight(weight, scale, x, K, "weight")
    b = 0 if bias is None else _vector(bias, x, N, x.dtype, "bias")
    if out is None:
        out, ldc = _empty(x, (M, N), x.dtype, stream), N if N > 0 else 1
    else:
        ldc = _like(x, out, M, N, x.dtype, "out")
    need = 0
    if K > 2048 and M <= 64 and workspace is not None:
        st, need = gemm_w4_bt_workspace_size(M, N, K)
        if st != GR_OK:
            raise GemmReluError(st, "gemm_w4_bt_workspace_size")
    ws, ws_bytes, keep = _scratch(x, need, workspace, stream)
    _run(_l.gemm_w4_bt, x, (M, N, K, x.data_ptr(), ldx, weight.data_ptr(), ldw, scale.data_ptr(), ldsw, b, _act(act),
                            out.data_ptr(), ldc, fmt, ws, ws_bytes), stream, "gemm_w4_bt")
    return out


def gemm_mxfp4(a, scale_a, bt, scale_b, bias=None, act="relu", out_dtype=None, out=None, stream=None, path=None):
    """``out = act(A @ B.T + bias)`` with both operands in MX fp4: ``a`` M x
    K/2 and ``bt`` N x K/2 uint8 (E2M1 pairs), ``scale_a`` M x K/32 and ``scale_b``
    N x K/32 uint8; fp16 or bfloat16 output as for gemm_mxfp8."""
    if _torch is None:
        _init()
    if a.dim() != 2:
        raise ValueError("a must be 2-D")
    if not a.is_cuda:
        raise ValueError("a must be a GPU tensor")
    K = a.shape[1] * 2
    M, lda, ldsa = _mxfp4_weight(a, scale_a, a, K, "a")
    N, ldbt, ldsb = _mxfp4_weight(bt, scale_b, a, K, "bt")
    if out is not None:
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = _torch.float16
    fmt = _FMT.get(out_dtype)
    if fmt is None:
        raise TypeError("the output is float16 or bfloat16")
    if out is None:
        out, ldc = _empty(a, (M, N), out_dtype, stream), N if N > 0 else 1
    else:
        ldc = _like(a, out, M, N, out_dtype, "out")
    b = 0 if bias is None else _vector(bias, a, N, out_dtype, "bias")
    args = (M, N, K, a.data_ptr(), lda, scale_a.data_ptr(), ldsa, bt.data_ptr(), ldbt, scale_b.data_ptr(), ldsb, b,
            _act(act), out.data_ptr(), ldc, fmt)
    if path is None:
        _run(_l.gemm_mxfp4_bt, a, args, stream, "gemm_mxfp4_bt")
    else:
        _run(lambda *v: gemm_mxfp4_bt_forced(*v, path), a, args, stream, "gemm_mxfp4_bt_forced")
    return out


def _scratch(x, need, workspace, stream):
    """(address, bytes) of a workspace: `need` bytes for "auto", the given tensor, or none."""
    if workspace is None or (workspace.__class__ is str and need == 0):
        return 0, 0, None
    if workspace.__class__ is str:
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', a uint8 tensor or None")
        workspace = _empty(x, (need,), _torch.uint8, stream)
    elif workspace.get_device() != x.get_device():
        raise ValueError("workspace is on another device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def moe_route(x, router, topk, bias=None, renormalize=True, workspace="auto", stream=None):
    """``(ids, weights)``, T x topk int32 and float32: the topk experts of each
    row of x (T x H) by ``x @ router.T + bias`` (router E x H in x's type, bias E
    float32), in descending order, and the softmax of their logits (over the
    chosen, or over all E with ``renormalize`` false).  ``workspace`` as for
    gemm_relu."""
    fmt, T, H, ldx = _matrix(x, "x")
    if router.dim() != 2:
        raise ValueError("router must be 2-D")
    E = router.shape[0]
    ldr = _like(x, router, E, H, x.dtype, "router")
    b = 0 if bias is None else _vector(bias, x, E, _torch.float32, "bias")
    k = topk if topk > 0 else 0
    need = 0
    if T * E * H > 65536 and workspace is not None:
        st, need = moe_route_workspace_size(T, H, E)
        if st != GR_OK:
            raise GemmReluError(st, "moe_route_workspace_size")
    ws, ws_bytes, keep = _scratch(x, need, workspace, stream)
    ids, weights = _empty(x, (T, k), _torch.int32, stream), _empty(x, (T, k), _torch.float32, stream)
    _run(_l.moe_route, x, (T, H, E, topk, x.data_ptr(), ldx, router.data_ptr(), ldr, b, 1 if renormalize else 0,
                           ids.data_ptr(), weights.data_ptr(), fmt, ws, ws_bytes), stream, "moe_route")
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
    for gemm_relu, but needed.
    """
    fmt, T, H, ldx = _matrix(x, "x")
    if ids.dtype != _torch.int32 or weights.dtype != _torch.float32:
        raise TypeError("ids must be int32 and weights float32")
    if ids.dim() != 2 or ids.shape[0] != T or ids.shape != weights.shape:
        raise ValueError("ids and weights must be %d x topk" % T)
    topk = ids.shape[1]
    if w13.dim() != 3 or w13.shape[1] % 2:
        raise ValueError("w13 must be E x 2I x H/2")
    E, I = w13.shape[0], w13.shape[1] // 2
    if H % 32 or I % 32:
        raise ValueError("H and I must be multiples of 32")
    device, u8 = x.get_device(), _torch.uint8
    for t, kind, shape in ((ids, _torch.int32, (T, topk)), (weights, _torch.float32, (T, topk)),
                           (w13, u8, (E, 2 * I, H // 2)), (s13, u8, (E, 2 * I, H // 32)), (w2, u8, (E, H, I // 2)),
                           (s2, u8, (E, H, I // 32)), (b13, x.dtype, (E, 2 * I)), (b2, x.dtype, (E, H))):
        if t is not None:
            if t.dtype != kind or t.shape != shape:
                raise ValueError("a tensor of the experts must be %s of %s, got %s of %s" % (shape, kind,
                                                                                            tuple(t.shape), t.dtype))
            if t.get_device() != device or not t.is_contiguous():
                raise ValueError("ids, weights, expert weights and biases must be contiguous and on x's device")
    if out is None:
        out, ldc = _empty(x, (T, H), x.dtype, stream), H if H > 0 else 1
    else:
        ldc = _like(x, out, T, H, x.dtype, "out")
    st, need = moe_w4_workspace_size(T, H, I, E, topk)
    if st != GR_OK:
        raise GemmReluError(st, "moe_w4_workspace_size")
    ws, ws_bytes, keep = _scratch(x, need, workspace, stream)
    if workspace is None and need > 0:
        raise GemmReluError(GR_ERR_SCRATCH, "moe_w4")
    _run(_l.moe_w4, x, (T, H, I, E, topk, x.data_ptr(), ldx, ids.data_ptr(), weights.data_ptr(), w13.data_ptr(),
                        s13.data_ptr(), 0 if b13 is None else b13.data_ptr(), w2.data_ptr(), s2.data_ptr(),
                        0 if b2 is None else b2.data_ptr(), _act(act), out.data_ptr(), ldc, fmt, ws, ws_bytes), stream,
         "moe_w4")
    return out
