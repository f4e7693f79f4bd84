"""CPU tests of the training operators: what the C calls and the tensor helpers refuse, sizes of workspaces, and the plain
forms that the GPU tests compare with."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import dense_gemm_epilogue_tiled_amd as gr
import train_ref

A = 1 << 20
DY, X, W, DX, DW, DB, WS, GU, C = (A << 16 | i << 40 for i in range(1, 10))
BIG = 1 << 40


def gated(M=8, I=48, H=50, x=X, ldx=None, w=W, ldw=None, b=DB, act=4, c=C, ldc=None, gu=GU, ldgu=None, fmt=1, ws=WS, size=BIG):
    return gr.gated_linear_bt(M, I, H, x, ldx or max(H, 1), w, ldw or max(H, 1), b, act, c, ldc or max(I, 1), gu,
                              ldgu or max(2 * I, 1), fmt, ws, size)


def linear(M=8, N=48, K=50, dy=DY, lddy=None, x=X, ldx=None, w=W, ldw=None, dx=DX, lddx=None, dw=DW, lddw=None, db=DB, fmt=1,
           ws=WS, size=BIG):
    k = max(K, 1)
    return gr.linear_backward_raw(M, N, K, dy, lddy or max(N, 1), x, ldx or k, w, ldw or k, dx, lddx or k, dw, lddw or k, db, fmt,
                                  ws, size)


def gated_bwd(M=8, I=24, H=50, dh=DY, lddh=None, x=X, ldx=None, w=W, ldw=None, gu=GU, ldgu=None, act=4, dx=DX, lddx=None, dw=DW,
              lddw=None, db=DB, fmt=1, ws=WS, size=BIG):
    h = max(H, 1)
    return gr.gated_linear_backward_raw(M, I, H, dh, lddh or max(I, 1), x, ldx or h, w, ldw or h, gu, ldgu or max(2 * I, 1), act,
                                        dx, lddx or h, dw, lddw or h, db, fmt, ws, size)


def norm(M=8, N=50, y=X, ldy=None, r=DY, ldr=None, w=W, next_w=DB, gate=GU, G=4, ldg=None, scale=1.0, eps=1e-6, total=DX,
         ldt=None, normed=DW, ldn=None, fmt=1):
    n = max(N, 1)
    return gr.sandwich_norm_fwd(M, N, y, ldy or n, r, ldr or n, w, next_w, gate, G, ldg or n, scale, eps, total, ldt or n, normed,
                                ldn or n, fmt)


def norm_bwd(M=8, N=50, dt=DY, dn=C, y=X, ldy=None, t=X + (1 << 30), w=W, next_w=W + 4096, gate=GU, G=4, ldg=None, scale=1.0,
             eps=1e-6, dy=DX, dr=DX + (1 << 30), dw=DW, dnext=DW + 4096, dgate=DB, ld_dgate=None, fmt=1, ws=WS, size=BIG):
    n = max(N, 1)
    return gr.sandwich_norm_bwd(M, N, dt, n, dn, n, y, ldy or n, t, n, w, next_w, gate, G, ldg or n, scale, eps, dy, n, dr, n, dw,
                                dnext, dgate, ld_dgate or n, fmt, ws, size)


def ortho(B=2, rows=150, cols=400, g=X, ldg=None, bg=None, g_fmt=2, k=train_ref.QUINTIC, steps=5, scale=1.0, eps=1e-7, out=C,
          ldo=None, bo=None, ws=WS, size=BIG):
    return gr.orthogonalize_update(B, rows, cols, g, ldg or max(cols, 1), rows * cols if bg is None else bg, g_fmt, k, steps, scale,
                                   eps, out, ldo or max(cols, 1), rows * cols if bo is None else bo, ws, size)


NAN, INF = float("nan"), float("inf")
REFUSALS = [
    (gated, dict(M=-1), gr.GR_ERR_INVALID_DIM), (gated, dict(I=1 << 31), gr.GR_ERR_TOO_LARGE),
    (gated, dict(I=1 << 30), gr.GR_ERR_TOO_LARGE), (gated, dict(ldx=49), gr.GR_ERR_INVALID_LD),
    (gated, dict(ldw=49), gr.GR_ERR_INVALID_LD), (gated, dict(ldc=47), gr.GR_ERR_INVALID_LD),
    (gated, dict(ldgu=95), gr.GR_ERR_INVALID_LD), (gated, dict(act=7), gr.GR_ERR_INVALID_ARG),
    (gated, dict(fmt=2), gr.GR_ERR_INVALID_ARG), (gated, dict(x=None), gr.GR_ERR_NULL_PTR), (gated, dict(w=None), gr.GR_ERR_NULL_PTR),
    (gated, dict(c=None), gr.GR_ERR_NULL_PTR), (gated, dict(ws=None, size=0), gr.GR_ERR_NULL_PTR),
    (gated, dict(size=255), gr.GR_ERR_SCRATCH), (gated, dict(ws=WS + 8), gr.GR_ERR_INVALID_ARG),
    (gated, dict(size=-1), gr.GR_ERR_INVALID_ARG), (gated, dict(c=X), gr.GR_ERR_ALIAS), (gated, dict(c=W + 2), gr.GR_ERR_ALIAS),
    (gated, dict(gu=C), gr.GR_ERR_ALIAS), (gated, dict(gu=DB), gr.GR_ERR_ALIAS), (gated, dict(ws=X), gr.GR_ERR_ALIAS),
    (gated, dict(ws=GU), gr.GR_ERR_ALIAS), (gated, dict(ldw=(1 << 22) + 1), gr.GR_ERR_TOO_LARGE),
    (linear, dict(K=-1), gr.GR_ERR_INVALID_DIM), (linear, dict(N=1 << 31), gr.GR_ERR_TOO_LARGE),
    (linear, dict(M=(1 << 22) + 1), gr.GR_ERR_TOO_LARGE), (linear, dict(lddy=47), gr.GR_ERR_INVALID_LD),
    (linear, dict(ldx=49), gr.GR_ERR_INVALID_LD), (linear, dict(ldw=49), gr.GR_ERR_INVALID_LD),
    (linear, dict(lddx=49), gr.GR_ERR_INVALID_LD), (linear, dict(lddw=49), gr.GR_ERR_INVALID_LD),
    (linear, dict(fmt=2), gr.GR_ERR_INVALID_ARG), (linear, dict(dy=None), gr.GR_ERR_NULL_PTR),
    (linear, dict(x=None), gr.GR_ERR_NULL_PTR), (linear, dict(w=None), gr.GR_ERR_NULL_PTR),
    (linear, dict(ws=None, size=0), gr.GR_ERR_NULL_PTR), (linear, dict(size=1000), gr.GR_ERR_SCRATCH),
    (linear, dict(ws=WS + 16), gr.GR_ERR_INVALID_ARG), (linear, dict(dx=X), gr.GR_ERR_ALIAS), (linear, dict(dx=DY), gr.GR_ERR_ALIAS),
    (linear, dict(dw=DX), gr.GR_ERR_ALIAS), (linear, dict(dw=W), gr.GR_ERR_ALIAS), (linear, dict(db=DX + 2), gr.GR_ERR_ALIAS),
    (linear, dict(ws=X), gr.GR_ERR_ALIAS), (linear, dict(ws=DW), gr.GR_ERR_ALIAS),
    (gated_bwd, dict(M=-1), gr.GR_ERR_INVALID_DIM), (gated_bwd, dict(I=1 << 30), gr.GR_ERR_TOO_LARGE),
    (gated_bwd, dict(M=(1 << 22) + 1), gr.GR_ERR_TOO_LARGE), (gated_bwd, dict(lddh=23), gr.GR_ERR_INVALID_LD),
    (gated_bwd, dict(ldgu=47), gr.GR_ERR_INVALID_LD), (gated_bwd, dict(lddw=49), gr.GR_ERR_INVALID_LD),
    (gated_bwd, dict(act=-1), gr.GR_ERR_INVALID_ARG), (gated_bwd, dict(fmt=9), gr.GR_ERR_INVALID_ARG),
    (gated_bwd, dict(gu=None), gr.GR_ERR_NULL_PTR), (gated_bwd, dict(dh=None), gr.GR_ERR_NULL_PTR),
    (gated_bwd, dict(x=None), gr.GR_ERR_NULL_PTR), (gated_bwd, dict(w=None), gr.GR_ERR_NULL_PTR),
    (gated_bwd, dict(size=1000), gr.GR_ERR_SCRATCH), (gated_bwd, dict(dw=GU), gr.GR_ERR_ALIAS),
    (gated_bwd, dict(dx=DY), gr.GR_ERR_ALIAS), (gated_bwd, dict(db=X), gr.GR_ERR_ALIAS), (gated_bwd, dict(ws=GU), gr.GR_ERR_ALIAS),
    (norm, dict(M=-1), gr.GR_ERR_INVALID_DIM), (norm, dict(N=32769), gr.GR_ERR_TOO_LARGE), (norm, dict(G=3), gr.GR_ERR_INVALID_DIM),
    (norm, dict(G=0), gr.GR_ERR_INVALID_DIM), (norm, dict(gate=None), gr.GR_ERR_INVALID_DIM), (norm, dict(ldy=49), gr.GR_ERR_INVALID_LD),
    (norm, dict(ldr=49), gr.GR_ERR_INVALID_LD), (norm, dict(ldg=49), gr.GR_ERR_INVALID_LD), (norm, dict(ldt=49), gr.GR_ERR_INVALID_LD),
    (norm, dict(ldn=49), gr.GR_ERR_INVALID_LD), (norm, dict(eps=-1.0), gr.GR_ERR_INVALID_ARG), (norm, dict(eps=NAN), gr.GR_ERR_INVALID_ARG),
    (norm, dict(scale=INF), gr.GR_ERR_INVALID_ARG), (norm, dict(fmt=2), gr.GR_ERR_INVALID_ARG), (norm, dict(y=None), gr.GR_ERR_NULL_PTR),
    (norm, dict(r=None), gr.GR_ERR_NULL_PTR), (norm, dict(total=None), gr.GR_ERR_NULL_PTR), (norm, dict(total=X + 2), gr.GR_ERR_ALIAS),
    (norm, dict(total=X, ldt=51), gr.GR_ERR_ALIAS), (norm, dict(normed=DX), gr.GR_ERR_ALIAS), (norm, dict(total=W), gr.GR_ERR_ALIAS),
    (norm, dict(normed=GU), gr.GR_ERR_ALIAS), (norm, dict(total=X, normed=X), gr.GR_ERR_ALIAS),
    (norm_bwd, dict(N=-1), gr.GR_ERR_INVALID_DIM), (norm_bwd, dict(G=3), gr.GR_ERR_INVALID_DIM),
    (norm_bwd, dict(N=32769), gr.GR_ERR_TOO_LARGE), (norm_bwd, dict(ldy=49), gr.GR_ERR_INVALID_LD),
    (norm_bwd, dict(ld_dgate=49), gr.GR_ERR_INVALID_LD), (norm_bwd, dict(dt=None, dn=None, dnext=None), gr.GR_ERR_NULL_PTR),
    (norm_bwd, dict(dn=None), gr.GR_ERR_INVALID_ARG), (norm_bwd, dict(gate=None, G=0), gr.GR_ERR_INVALID_ARG),
    (norm_bwd, dict(y=None), gr.GR_ERR_NULL_PTR), (norm_bwd, dict(t=None), gr.GR_ERR_NULL_PTR), (norm_bwd, dict(dy=None), gr.GR_ERR_NULL_PTR),
    (norm_bwd, dict(dr=None), gr.GR_ERR_NULL_PTR), (norm_bwd, dict(ws=None, size=0), gr.GR_ERR_NULL_PTR),
    (norm_bwd, dict(size=64), gr.GR_ERR_SCRATCH), (norm_bwd, dict(dy=DY), gr.GR_ERR_ALIAS), (norm_bwd, dict(dr=DX), gr.GR_ERR_ALIAS),
    (norm_bwd, dict(dw=W), gr.GR_ERR_ALIAS), (norm_bwd, dict(dgate=DW), gr.GR_ERR_ALIAS), (norm_bwd, dict(ws=X), gr.GR_ERR_ALIAS),
    (ortho, dict(B=-1), gr.GR_ERR_INVALID_DIM), (ortho, dict(B=65536), gr.GR_ERR_TOO_LARGE), (ortho, dict(rows=65537), gr.GR_ERR_TOO_LARGE),
    (ortho, dict(cols=1 << 31), gr.GR_ERR_TOO_LARGE), (ortho, dict(ldg=399), gr.GR_ERR_INVALID_LD), (ortho, dict(ldo=399), gr.GR_ERR_INVALID_LD),
    (ortho, dict(bg=59999), gr.GR_ERR_INVALID_LD), (ortho, dict(bo=-1), gr.GR_ERR_INVALID_LD), (ortho, dict(bg=1 << 60), gr.GR_ERR_TOO_LARGE),
    (ortho, dict(g_fmt=3), gr.GR_ERR_INVALID_ARG), (ortho, dict(steps=0), gr.GR_ERR_INVALID_ARG), (ortho, dict(steps=65), gr.GR_ERR_INVALID_ARG),
    (ortho, dict(k=(1.0, NAN, 1.0)), gr.GR_ERR_INVALID_ARG), (ortho, dict(scale=NAN), gr.GR_ERR_INVALID_ARG),
    (ortho, dict(eps=-1.0), gr.GR_ERR_INVALID_ARG), (ortho, dict(g=None), gr.GR_ERR_NULL_PTR), (ortho, dict(out=None), gr.GR_ERR_NULL_PTR),
    (ortho, dict(ws=None, size=0), gr.GR_ERR_NULL_PTR), (ortho, dict(size=1 << 16), gr.GR_ERR_SCRATCH), (ortho, dict(out=X + 4), gr.GR_ERR_ALIAS),
    (ortho, dict(ws=C), gr.GR_ERR_ALIAS),
]


@pytest.mark.parametrize("call,args,status", REFUSALS, ids=lambda v: v.__name__ if callable(v) else str(v)[:40])
def test_refused(call, args, status):
    assert call(**args) == status


@pytest.mark.parametrize("call,args", [
    (gated, dict(M=0, x=None, c=None, gu=None)), (gated, dict(I=0, w=None, c=None, gu=None, b=None)),
    (linear, dict(M=0, K=0, N=0, db=None)), (gated_bwd, dict(dx=None, dw=None, db=None)), (norm, dict(M=0, G=1, y=None)),
    (norm, dict(N=0)), (norm_bwd, dict(N=0)), (norm_bwd, dict(M=0, dw=None, dnext=None, dgate=None)), (ortho, dict(B=0, g=None)),
    (ortho, dict(rows=0, out=None)), (ortho, dict(cols=0))])
def test_empty_is_ok_without_a_device(call, args):
    if call is linear:
        args = dict(args, dx=None, dw=None)
    assert call(**args) in ((gr.GR_OK,) if call is not linear else (gr.GR_OK, gr.GR_ERR_NO_DEVICE))


def test_valid_calls_get_as_far_as_the_device():
    if torch.cuda.is_available():
        pytest.skip("there is a device, and these pointers are none of its")
    for call in (gated, linear, gated_bwd, norm, norm_bwd, ortho):
        assert call() == gr.GR_ERR_NO_DEVICE, call
    assert norm(total=X, normed=DY) == norm(total=DY, normed=X) == gr.GR_ERR_NO_DEVICE
    assert ortho(rows=100, cols=300, ws=None, size=0) == gr.GR_ERR_NO_DEVICE  # small: no workspace
    assert gated(H=64, ws=None, size=0) == gated(M=4, ws=None, size=0) == gr.GR_ERR_NO_DEVICE


def test_workspace_sizes():
    assert gr.gated_linear_workspace_size(100, 48, 64) == (gr.GR_OK, 0)
    assert gr.gated_linear_workspace_size(4, 48, 50) == (gr.GR_OK, 0)
    assert gr.gated_linear_workspace_size(100, 48, 50) == (gr.GR_OK, 100 * 128 + 96 * 128)
    assert gr.gated_linear_workspace_size(-1, 48, 50)[0] == gr.GR_ERR_INVALID_DIM

    def linear_size(dx=DX, dw=DW, db=DB, M=100):
        return gr.linear_backward_workspace_size(M, 48, 50, DY, 48, X, 50, W, 50, dx, 50, dw, 50, db)

    st, whole = linear_size()
    assert st == gr.GR_OK and whole % 256 == 0 and whole >= 128 * 2 * (48 + 50)
    assert linear_size(dx=None)[1] < whole and linear_size(dw=None, db=None)[1] < whole
    assert linear_size(None, None, None) == (gr.GR_OK, 0)
    assert linear_size(M=-1)[0] == gr.GR_ERR_INVALID_DIM
    st, n = gr.gated_linear_backward_workspace_size(100, 24, 50, W, 50, DX, 50, DW, DB)
    assert st == gr.GR_OK and n % 256 == 0 and n >= 128 * 2 * (48 + 50) + 100 * 2 * 48
    assert gr.sandwich_norm_bwd_workspace_size(8, 64, 4)[1] >= 4 * 2 * 64 * 4
    assert gr.sandwich_norm_bwd_workspace_size(8, 64, 3)[0] == gr.GR_ERR_INVALID_DIM
    assert gr.orthogonalize_workspace_size(1, 128, 512) == gr.orthogonalize_workspace_size(5, 512, 100) == (gr.GR_OK, 0)
    st, n = gr.orthogonalize_workspace_size(1, 4096, 8192)
    assert st == gr.GR_OK and n >= 2 * (4 * 4096 * 8192 + 2 * 4096 * 4096)
    assert gr.orthogonalize_workspace_size(0, 8, 8) == (gr.GR_OK, 0)
    none = ctypes.POINTER(ctypes.c_int64)()
    assert gr.lib().gated_linear_workspace_size(1, 2, 3, none) == gr.GR_ERR_INVALID_ARG
    assert gr.lib().orthogonalize_workspace_size(1, 2, 3, none) == gr.GR_ERR_INVALID_ARG


# ---- tensor helpers --------------------------------------------------------------------

def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def helpers():
    gr.lib()
    from dense_gemm_epilogue_tiled_amd import _tensors
    return _tensors


def h_gated(x=None, w=None, b=None, out=None, gu=None, keep=1):
    return helpers().gated_linear(zeros(4, 32) if x is None else x, zeros(16, 32) if w is None else w, b, 4, keep, out, gu, None, 0)


def h_linear(dy=None, x=zeros(4, 32), w=None, dx=None, dw=None, want=1):
    return helpers().linear_backward(zeros(4, 8) if dy is None else dy, x, zeros(8, 32) if w is None else w, 1, want, want, dx, dw,
                                     None, 0)


def h_gated_bwd(dh=None, x=zeros(4, 32), w=None, gu=None, dx=None, dw=None):
    return helpers().gated_linear_backward(zeros(4, 8) if dh is None else dh, x, zeros(16, 32) if w is None else w,
                                           zeros(4, 16) if gu is None else gu, 4, 1, 1, 1, dx, dw, None, 0)


def h_norm(y=None, r=None, w=None, next_w=None, gate=None, total=None, normed=None, norm=1):
    return helpers().sandwich_norm(zeros(4, 32) if y is None else y, zeros(4, 32) if r is None else r, w, next_w, gate, 1.0, 1e-6,
                                   norm, total, normed, 0)


def h_norm_bwd(y=None, dt=zeros(4, 32), dn=None, t=None, w=None, next_w=None, gate=None):
    return helpers().sandwich_norm_backward(zeros(4, 32) if y is None else y, dt, dn, zeros(4, 32) if t is None else t, w, next_w,
                                            gate, 1.0, 1e-6, None, 0)


def h_ortho(g=None, out=None):
    return helpers().orthogonalize(zeros(2, 8, 32) if g is None else g, 5, 1.0, 1.0, 1.0, 1.0, 1e-7, out, None, 0)


HELPERS = [h_gated, h_linear, h_gated_bwd, h_norm, h_norm_bwd, h_ortho]
half = zeros(4, 32, dtype=torch.float16)
one_row = zeros(1, 32).expand(4, 32)


@pytest.mark.parametrize("call", HELPERS)
def test_cpu_tensors_are_refused(call):
    with pytest.raises(ValueError, match="GPU"):
        call()


BAD = [(h_gated, dict(x=zeros(4, 31))), (h_gated, dict(w=zeros(15, 32))), (h_gated, dict(b=zeros(15))),
       (h_gated, dict(out=zeros(4, 9))), (h_gated, dict(gu=zeros(4, 16), keep=0, out=zeros(4, 8))), (h_gated, dict(x=one_row)),
       (h_gated, dict(x=zeros(32, 4).T)), (h_gated, dict(out=zeros(1, 8).expand(4, 8))),
       (h_linear, dict(x=zeros(4, 31))), (h_linear, dict(x=None)), (h_linear, dict(w=zeros(9, 32))), (h_linear, dict(dx=zeros(4, 33))),
       (h_linear, dict(dx=zeros(4, 32), dw=zeros(8, 64)[:, ::2])), (h_linear, dict(dx=zeros(4, 32), want=0)), (h_linear, dict(x=half)),
       (h_gated_bwd, dict(w=zeros(18, 32))), (h_gated_bwd, dict(gu=zeros(4, 15))), (h_gated_bwd, dict(x=None)),
       (h_gated_bwd, dict(gu=half[:, :16])), (h_gated_bwd, dict(dw=zeros(16, 31), dx=zeros(4, 32))),
       (h_norm, dict(r=zeros(4, 31))), (h_norm, dict(r=half)), (h_norm, dict(w=zeros(31))), (h_norm, dict(w=zeros(64)[::2])),
       (h_norm, dict(gate=zeros(3, 32))), (h_norm, dict(gate=zeros(0, 32))), (h_norm, dict(gate=zeros(1, 2, 32))),
       (h_norm, dict(gate=zeros(31))), (h_norm, dict(total=zeros(4, 31))), (h_norm, dict(next_w=zeros(32), norm=0)),
       (h_norm, dict(y=one_row)), (h_norm_bwd, dict(dt=None)), (h_norm_bwd, dict(t=zeros(3, 32))), (h_norm_bwd, dict(dn=zeros(4, 31))),
       (h_norm_bwd, dict(gate=zeros(8, 32))), (h_ortho, dict(g=zeros(8))), (h_ortho, dict(g=zeros(2, 32, 8).transpose(1, 2))),
       (h_ortho, dict(g=zeros(1, 8, 32).expand(2, 8, 32))), (h_ortho, dict(g=one_row)), (h_ortho, dict(out=zeros(2, 8, 31))),
       (h_ortho, dict(out=zeros(2, 8, 32, dtype=torch.float32))), (h_ortho, dict(out=zeros(1, 8, 32).expand(2, 8, 32)))]


@pytest.mark.parametrize("call,args", BAD, ids=lambda v: v.__name__ if callable(v) else "-".join(v))
def test_helpers_refuse(call, args):
    with pytest.raises(ValueError) as e:
        call(**args)
    assert "GPU tensor" not in str(e.value)


@pytest.mark.parametrize("call,args", [(h_gated, dict(x=zeros(4, 32, dtype=torch.float32))), (h_gated, dict(x=half)),
                                       (h_linear, dict(dy=zeros(4, 8, dtype=torch.int32))), (h_linear, dict(w=half[:, :32].repeat(2, 1))),
                                       (h_gated_bwd, dict(w=half.repeat(4, 1))), (h_norm, dict(y=zeros(4, 32, dtype=torch.float64))),
                                       (h_ortho, dict(g=zeros(4, 4, dtype=torch.float64))), (h_norm, dict(r=3)), (h_ortho, dict(g=None, out=1))])
def test_helpers_refuse_types(call, args):
    with pytest.raises(TypeError):
        call(**args)


def wants(*shape, dtype=torch.bfloat16):
    return zeros(*shape, dtype=dtype).requires_grad_()


@pytest.mark.parametrize("call,args", [(h_gated, lambda: dict(x=wants(4, 32))), (h_gated, lambda: dict(w=wants(16, 32))),
                                       (h_gated, lambda: dict(b=wants(16))), (h_linear, lambda: dict(x=wants(4, 32))),
                                       (h_gated_bwd, lambda: dict(gu=wants(4, 16))), (h_norm, lambda: dict(gate=wants(2, 32))),
                                       (h_norm_bwd, lambda: dict(next_w=wants(32))), (h_ortho, lambda: dict(g=wants(8, 8)))])
def test_recorded_gradients_are_refused(call, args):
    """Nothing is recorded for autograd: a tensor whose gradient would be lost is refused, unless nothing is recorded."""
    with pytest.raises(RuntimeError, match="no gradient"):
        call(**args())
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        call(**args())


def test_kernels_keep_to_registers():
    """The products' kernels do not spill, and no other kernel does but the norms' backward passes of rows above 8192 columns
    and of more gates than workgroups, and the small matrices' kernel, whose spills lie outside its loops over k."""
    from dense_gemm_epilogue_tiled_amd import build as b
    for unit in ("train_ops.hip", "update_ops.hip"):
        cmd = [b.HIPCC, *b.FLAGS, "-c", "--cuda-device-only", os.path.join(b.HERE, "csrc", unit), "-o", os.devnull,
               "-Rpass-analysis=kernel-resource-usage"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-2000:]
        names = re.findall(r"Function Name: (\S+)", res.stderr)
        scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", res.stderr)]
        assert names and len(names) == len(scratch)
        for n, s in zip(names, scratch):
            wide = re.search(r"backward_kernelI\w+?Li(\d+)ELi(\d+)ELb(\d)", n)
            if "sandwich" in n and wide and (int(wide[2]) > 1 or wide[3] == "0"):
                continue
            assert s <= (128 if "small_kernel" in n else 0), (n, s)


# ---- the plain forms -----------------------------------------------------------------------

def test_plain_slopes_are_derivatives():
    v = torch.linspace(-9, 9, 1801, dtype=torch.float64) + 1e-3
    for name in ("relu", "gelu", "gelu_tanh", "silu", "sigmoid", "tanh", "none"):
        e = 1e-6
        quotient = (train_ref.act(v + e, name) - train_ref.act(v - e, name)) / (2 * e)
        assert float((quotient - train_ref.slope(v, name)).abs().max()) < 1e-8, name


def test_plain_gradients_are_autograds():
    g = torch.Generator().manual_seed(1)

    def rand(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)

    y, res, w, w2, gate, dt, dn = rand(6, 9), rand(6, 9), rand(9), rand(9), rand(3, 9), rand(6, 9), rand(6, 9)
    leaves = [t.clone().requires_grad_() for t in (y, res, w, w2, gate)]
    total, _, _ = train_ref.sandwich(*leaves[:3], leaves[3], leaves[4], 0.7, 1e-3)
    normed = train_ref.next_norm(total, leaves[3], 1e-3)
    want = torch.autograd.grad((total * dt).sum() + (normed * dn).sum(), leaves)
    got = train_ref.sandwich_backward(dt, dn, y, total.detach(), w, w2, gate, 0.7, 1e-3)
    for (value, _), grad in zip(got.values(), want):
        assert torch.allclose(value, grad, rtol=1e-9, atol=1e-12)
    x, w13, dh = rand(5, 7), rand(8, 7), rand(5, 4).bfloat16()
    a, b = x.clone().requires_grad_(), w13.clone().requires_grad_()
    gu = a @ b.T
    want = torch.autograd.grad((train_ref.act(gu[:, :4], "gelu") * gu[:, 4:] * dh.double()).sum(), (a, b))
    got, _ = train_ref.gated_backward(dh, x, w13, gu.detach(), "gelu")
    for value, grad in zip(got, want):
        assert torch.allclose(value, grad, rtol=1e-9, atol=1e-12)


def test_plain_newton_schulz_is_the_polynomial_of_the_singular_values():
    x = torch.randn(5, 8, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    u, s, vh = torch.linalg.svd(x, full_matrices=False)
    s = s / (s.square().sum().sqrt() + 1e-7)
    a, b, c = train_ref.QUINTIC
    for _ in range(4):
        s = a * s + b * s ** 3 + c * s ** 5
    want = (u * s) @ vh
    assert torch.allclose(train_ref.newton_schulz(x, 4), want, rtol=1e-9, atol=1e-12)
    assert torch.allclose(train_ref.newton_schulz(x.T, 4), want.T, rtol=1e-9, atol=1e-12)
