"""Argument checks of the operators around the MX products (no GPU needed), and pins of the tests' own plain forms."""
import ctypes

import pytest
import torch

import dense_gemm_epilogue_tiled_amd as gr
import mx_ref

X, R, W, S, Y, SY, B, I = (0x100000000000 + i * 0x10000000000 for i in range(8))
BF, F16 = gr.GR_FMT_BF16, gr.GR_FMT_F16


def norm(M=4, N=64, x=X, ldx=64, r=R, ldr=64, w=W, eps=1e-6, s=S, lds=64, y=Y, ldy=64, sy=SY, ld_sy=2, fmt=BF,
         out=gr.GR_OUT_MXFP8):
    return gr.rms_norm_mx(M, N, x, ldx, r, ldr, w, eps, s, lds, y, ldy, sy, ld_sy, fmt, out)


def gated(M=4, N=64, g=X, ldg=64, u=R, ldu=64, act=gr.GR_ACT_SILU, y=Y, ldy=64, sy=SY, ld_sy=2, fmt=BF,
          out=gr.GR_OUT_MXFP8):
    return gr.gated_act_mx(M, N, g, ldg, u, ldu, act, y, ldy, sy, ld_sy, fmt, out)


WS = 0x900000000000


def linear(M=4, N=48, K=64, a=X, lda=64, bt=W, ldbt=32, s=S, lds=2, bias=None, act=gr.GR_ACT_NONE, c=Y, ldc=48,
           fmt=BF, ws=None, size=0):
    return gr.gemm_w4_bt(M, N, K, a, lda, bt, ldbt, s, lds, bias, act, c, ldc, fmt, ws, size)


def fp4(M=4, N=48, K=64, a=X, lda=32, sa=R, ld_sa=2, bt=W, ldbt=32, s=S, lds=2, bias=None, act=gr.GR_ACT_NONE, c=Y,
        ldc=48, fmt=BF):
    return gr.gemm_mxfp4_linear_bt(M, N, K, a, lda, sa, ld_sa, bt, ldbt, s, lds, bias, act, c, ldc, fmt)


def route(T=4, H=64, E=8, k=2, x=X, ldx=64, w=W, ldw=64, bias=None, renorm=1, ids=I, weights=Y, fmt=BF, ws=None,
          size=0):
    return gr.moe_route_raw(T, H, E, k, x, ldx, w, ldw, bias, renorm, ids, weights, fmt, ws, size)


def moe(T=4, H=64, I_=96, E=8, k=2, x=X, ldx=64, ids=I, weights=R, w13=W, s13=S, b13=None, w2=B, s2=SY, b2=None,
        act=gr.GR_ACT_SILU, c=Y, ldc=64, fmt=BF, ws=0x900000000000, size=None):
    if size is None:
        size = 4 * max(T, 0) * (max(I_, 0) + max(H, 0) + 1) * max(k, 0) + 768
    return gr.moe_w4(T, H, I_, E, k, x, ldx, ids, weights, w13, s13, b13, w2, s2, b2, act, c, ldc, fmt, ws, size)


REFUSALS = [
    (norm, dict(M=-1), gr.GR_ERR_INVALID_DIM),
    (norm, dict(N=48, ldx=48, ldr=48, lds=48), gr.GR_ERR_INVALID_DIM),
    (norm, dict(M=1 << 31), gr.GR_ERR_TOO_LARGE),
    (norm, dict(ldx=63), gr.GR_ERR_INVALID_LD),
    (norm, dict(ldr=63), gr.GR_ERR_INVALID_LD),
    (norm, dict(lds=63), gr.GR_ERR_INVALID_LD),
    (norm, dict(ldy=63), gr.GR_ERR_INVALID_LD),
    (norm, dict(ldy=31, out=gr.GR_OUT_MXFP4), gr.GR_ERR_INVALID_LD),
    (norm, dict(ld_sy=1), gr.GR_ERR_INVALID_LD),
    (norm, dict(x=None), gr.GR_ERR_NULL_PTR),
    (norm, dict(y=None), gr.GR_ERR_NULL_PTR),
    (norm, dict(sy=None), gr.GR_ERR_NULL_PTR),
    (norm, dict(eps=-1.0), gr.GR_ERR_INVALID_ARG),
    (norm, dict(eps=float("nan")), gr.GR_ERR_INVALID_ARG),
    (norm, dict(eps=float("inf")), gr.GR_ERR_INVALID_ARG),
    (norm, dict(fmt=2), gr.GR_ERR_INVALID_ARG),
    (norm, dict(out=3), gr.GR_ERR_INVALID_ARG),
    (norm, dict(r=None), gr.GR_ERR_INVALID_ARG),
    (norm, dict(s=X + 2), gr.GR_ERR_ALIAS),
    (norm, dict(s=X, lds=72), gr.GR_ERR_ALIAS),
    (norm, dict(y=X), gr.GR_ERR_ALIAS),
    (norm, dict(y=R, out=gr.GR_OUT_16), gr.GR_ERR_ALIAS),
    (norm, dict(y=S), gr.GR_ERR_ALIAS),
    (norm, dict(y=W), gr.GR_ERR_ALIAS),
    (norm, dict(sy=Y + 64), gr.GR_ERR_ALIAS),
    (norm, dict(r=X + 64, s=X), gr.GR_ERR_ALIAS),
    (gated, dict(N=40, ldg=64), gr.GR_ERR_INVALID_DIM),
    (gated, dict(N=-32), gr.GR_ERR_INVALID_DIM),
    (gated, dict(ldg=32), gr.GR_ERR_INVALID_LD),
    (gated, dict(ldu=32), gr.GR_ERR_INVALID_LD),
    (gated, dict(act=7), gr.GR_ERR_INVALID_ARG),
    (gated, dict(act=-1), gr.GR_ERR_INVALID_ARG),
    (gated, dict(out=-1), gr.GR_ERR_INVALID_ARG),
    (gated, dict(g=None), gr.GR_ERR_NULL_PTR),
    (gated, dict(y=X), gr.GR_ERR_ALIAS),
    (gated, dict(y=X + 2, out=gr.GR_OUT_16), gr.GR_ERR_ALIAS),
    (gated, dict(sy=R), gr.GR_ERR_ALIAS),
    (linear, dict(K=48), gr.GR_ERR_INVALID_DIM),
    (linear, dict(M=-1), gr.GR_ERR_INVALID_DIM),
    (linear, dict(N=1 << 31), gr.GR_ERR_TOO_LARGE),
    (linear, dict(lda=63), gr.GR_ERR_INVALID_LD),
    (linear, dict(ldbt=31), gr.GR_ERR_INVALID_LD),
    (linear, dict(lds=1), gr.GR_ERR_INVALID_LD),
    (linear, dict(ldc=47), gr.GR_ERR_INVALID_LD),
    (linear, dict(act=9), gr.GR_ERR_INVALID_ARG),
    (linear, dict(fmt=5), gr.GR_ERR_INVALID_ARG),
    (linear, dict(a=None), gr.GR_ERR_NULL_PTR),
    (linear, dict(s=None), gr.GR_ERR_NULL_PTR),
    (linear, dict(c=X), gr.GR_ERR_ALIAS),
    (linear, dict(c=W), gr.GR_ERR_ALIAS),
    (linear, dict(bias=Y), gr.GR_ERR_ALIAS),
    (linear, dict(ldbt=(1 << 26) + 1), gr.GR_ERR_TOO_LARGE),
    (linear, dict(ws=WS + 8, size=1 << 20), gr.GR_ERR_INVALID_ARG),
    (linear, dict(ws=WS, size=-1), gr.GR_ERR_INVALID_ARG),
    (linear, dict(M=64, K=8192, lda=8192, ldbt=4096, lds=256, ws=Y, size=1 << 30), gr.GR_ERR_ALIAS),
    (linear, dict(M=64, K=8192, lda=8192, ldbt=4096, lds=256, ws=W, size=1 << 30), gr.GR_ERR_ALIAS),
    (fp4, dict(K=48), gr.GR_ERR_INVALID_DIM),
    (fp4, dict(M=-1), gr.GR_ERR_INVALID_DIM),
    (fp4, dict(lda=31), gr.GR_ERR_INVALID_LD),
    (fp4, dict(ld_sa=1), gr.GR_ERR_INVALID_LD),
    (fp4, dict(ldbt=31), gr.GR_ERR_INVALID_LD),
    (fp4, dict(lds=1), gr.GR_ERR_INVALID_LD),
    (fp4, dict(ldc=47), gr.GR_ERR_INVALID_LD),
    (fp4, dict(act=9), gr.GR_ERR_INVALID_ARG),
    (fp4, dict(fmt=5), gr.GR_ERR_INVALID_ARG),
    (fp4, dict(a=None), gr.GR_ERR_NULL_PTR),
    (fp4, dict(sa=None), gr.GR_ERR_NULL_PTR),
    (fp4, dict(bt=None), gr.GR_ERR_NULL_PTR),
    (fp4, dict(c=None), gr.GR_ERR_NULL_PTR),
    (fp4, dict(c=X), gr.GR_ERR_ALIAS),
    (fp4, dict(c=S), gr.GR_ERR_ALIAS),
    (fp4, dict(bias=Y), gr.GR_ERR_ALIAS),
    (route, dict(k=0), gr.GR_ERR_INVALID_ARG),
    (route, dict(k=9), gr.GR_ERR_INVALID_ARG),
    (route, dict(E=0), gr.GR_ERR_INVALID_DIM),
    (route, dict(E=1025), gr.GR_ERR_TOO_LARGE),
    (route, dict(E=64, k=33), gr.GR_ERR_TOO_LARGE),
    (route, dict(renorm=2), gr.GR_ERR_INVALID_ARG),
    (route, dict(ldw=63), gr.GR_ERR_INVALID_LD),
    (route, dict(ids=None), gr.GR_ERR_NULL_PTR),
    (route, dict(ids=Y), gr.GR_ERR_ALIAS),
    (route, dict(weights=X), gr.GR_ERR_ALIAS),
    (route, dict(ws=WS + 4, size=1 << 20), gr.GR_ERR_INVALID_ARG),
    (route, dict(ws=WS, size=-5), gr.GR_ERR_INVALID_ARG),
    (route, dict(H=8192, E=64, ldx=8192, ldw=8192, ws=W, size=1 << 30), gr.GR_ERR_ALIAS),
    (moe, dict(H=48), gr.GR_ERR_INVALID_DIM),
    (moe, dict(I_=100), gr.GR_ERR_INVALID_DIM),
    (moe, dict(E=0), gr.GR_ERR_INVALID_DIM),
    (moe, dict(E=1025), gr.GR_ERR_TOO_LARGE),
    (moe, dict(k=33), gr.GR_ERR_TOO_LARGE),
    (moe, dict(I_=(1 << 20) + 32), gr.GR_ERR_TOO_LARGE),
    (moe, dict(k=0), gr.GR_ERR_INVALID_ARG),
    (moe, dict(ldx=63), gr.GR_ERR_INVALID_LD),
    (moe, dict(ids=None), gr.GR_ERR_NULL_PTR),
    (moe, dict(w2=None), gr.GR_ERR_NULL_PTR),
    (moe, dict(ws=None), gr.GR_ERR_NULL_PTR),
    (moe, dict(ws=0x900000000080), gr.GR_ERR_INVALID_ARG),
    (moe, dict(size=-1), gr.GR_ERR_INVALID_ARG),
    (moe, dict(size=256), gr.GR_ERR_SCRATCH),
    (moe, dict(c=X), gr.GR_ERR_ALIAS),
    (moe, dict(ws=W), gr.GR_ERR_ALIAS),
]


@pytest.mark.parametrize("call,args,status", REFUSALS, ids=lambda v: v.__name__ if callable(v) else str(v)[:40])
def test_refused(call, args, status):
    assert call(**args) == status


@pytest.mark.parametrize("call,args", [
    (norm, dict(M=0)), (norm, dict(N=0, x=None, y=None)), (gated, dict(M=0, g=None)), (gated, dict(N=0)),
    (linear, dict(M=0)), (linear, dict(N=0, ldc=1)), (fp4, dict(M=0)), (fp4, dict(N=0, ldc=1)), (route, dict(T=0)), (moe, dict(T=0)), (moe, dict(H=0))])
def test_empty_is_ok_without_a_device(call, args):
    assert call(**args) == gr.GR_OK


def test_workspace_size():
    st, n = gr.moe_w4_workspace_size(5, 64, 96, 8, 2)
    assert st == gr.GR_OK and n % 256 == 0 and n >= 5 * 2 * 96 * 4
    assert gr.moe_w4_workspace_size(0, 64, 96, 8, 2) == (gr.GR_OK, 0)
    assert gr.moe_w4_workspace_size(5, 64, 90, 8, 2)[0] == gr.GR_ERR_INVALID_DIM
    assert gr.lib().moe_w4_workspace_size(5, 64, 96, 8, 2, ctypes.POINTER(ctypes.c_int64)()) == gr.GR_ERR_INVALID_ARG


def test_workspace_sizes_of_the_products_and_the_router():
    """None where it would not help; the split sums' size where it does."""
    assert gr.gemm_w4_bt_workspace_size(1, 4096, 4096) == (gr.GR_OK, 0)
    st, n = gr.gemm_w4_bt_workspace_size(64, 8192, 8192)
    assert st == gr.GR_OK and n >= 2 * 64 * 8192 * 4 and n % 256 == 0
    assert gr.gemm_w4_bt_workspace_size(65, 8192, 8192) == (gr.GR_OK, 0)
    assert gr.gemm_w4_bt_workspace_size(0, 8192, 8192) == gr.gemm_w4_bt_workspace_size(4, 0, 8192) == (gr.GR_OK, 0)
    assert gr.gemm_w4_bt_workspace_size(4, 16, 0) == (gr.GR_OK, 0)
    assert gr.gemm_w4_bt_workspace_size(4, 16, 40)[0] == gr.GR_ERR_INVALID_DIM
    assert gr.moe_route_workspace_size(1, 64, 8) == (gr.GR_OK, 0)
    st, n = gr.moe_route_workspace_size(3, 4096, 64)
    assert st == gr.GR_OK and n >= 8 * 3 * 64 * 4
    assert gr.moe_route_workspace_size(100000, 4096, 64) == (gr.GR_OK, 0)
    assert gr.moe_route_workspace_size(1, 64, 0)[0] == gr.GR_ERR_INVALID_DIM


def test_streaming_kernels_keep_to_registers():
    """At most 16 registers of any kernel are spilled (the streaming kernels' spills surround their loops; a reload
    within waits for every load in flight): checked with the compiler's resource report."""
    import os
    import re
    import subprocess
    from dense_gemm_epilogue_tiled_amd import build as b
    unit = os.path.join(b.HERE, "csrc", "mx_ops.hip")
    cmd = [b.HIPCC, *b.FLAGS, "-c", "--cuda-device-only", unit, "-o", os.devnull,
           "-Rpass-analysis=kernel-resource-usage"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    names = re.findall(r"Function Name: (\S+)", res.stderr)
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", res.stderr)]
    assert names and len(names) == len(scratch)
    for n, s in zip(names, scratch):
        assert s <= 64, (n, s)


def test_helpers_refuse():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    for call in (lambda: gr.rms_norm(x), lambda: gr.gated_act(x), lambda: gr.linear_mxfp4(x, w, s),
                 lambda: gr.mx_quantize(x), lambda: gr.moe_route(x, x, 1)):
        with pytest.raises(ValueError):  # not a GPU tensor
            call()
    with pytest.raises(ValueError):
        gr.mx_quantize(x, "same")


# ---- the plain forms the GPU tests compare with ---------------------------------------

def test_plain_e2m1_rounds_to_nearest_even():
    a = torch.tensor([0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 6.0, 7.9], dtype=torch.float64)
    y = torch.zeros(1, 32, dtype=torch.float64)
    y[0, :12], y[0, 12:24] = a, -a
    q, e = mx_ref.quantise(y, "mxfp4")
    want = torch.tensor([0, 0, 0.5, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 6.0], dtype=torch.float64)
    assert int(e) == 0 and torch.equal(q[0, :12], want) and torch.equal(q[0, 12:24], -want)


def test_plain_e4m3_matches_torch_cast():
    g = torch.Generator().manual_seed(3)
    y = torch.randn(64, 32, generator=g).double() * 100
    y[:, 0] = 300.0  # exponent 8: scale 1
    y = y.clamp(-448, 448)
    q, e = mx_ref.quantise(y, "mxfp8")
    assert bool((e == 0).all())
    assert torch.equal(q, y.float().to(torch.float8_e4m3fn).double())


def test_plain_unpack():
    w = torch.tensor([[0x21, 0xF8]], dtype=torch.uint8)
    assert mx_ref.unpack4(w).tolist() == [[0.5, 1.0, -0.0, -6.0]]
