"""GPU parity of the operators around the MX products with their plain fp64 forms (mx_ref).

Bounds count roundings: half a step of the output type for the one rounding
at the end, and a few half steps of fp32 for the arithmetic before it, stated at
each test.
"""
import pytest
import torch

import dense_gemm_epilogue_tiled_amd as gr
import mx_ref
from gpu_util import log

pytestmark = pytest.mark.gpu

U = mx_ref.U32
# fp32 roundings of the RMS norm, relative: the sum of squares (at most 64 in a
# row and a tree of 12, halved by the root) and 5 more operations
NORM = 48 * U


def padded(x, pitch, offset=0, fill=None):
    """x on the GPU inside a larger buffer: row pitch `pitch`, first element at `offset`; (buffer, view)."""
    rows, cols = x.shape
    buf = torch.empty(rows * pitch + offset + 64, dtype=x.dtype, device="cuda")
    buf.view(torch.uint8).fill_(0x7F if fill is None else fill)
    view = buf[offset:offset + rows * pitch].view(rows, pitch)[:, :cols]
    view.copy_(x)
    return buf, view


def inputs(M, N, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, N, generator=g) * scale).to(mx_ref.TYPES[dtype])


# ---- RMS norm -----------------------------------------------------------------------

def norm_ref(x, r, w, eps):
    s = x if r is None else (x.float() + r.float()).to(x.dtype)
    v = s.double()
    y = v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
    return s, y if w is None else y * w.double()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["same", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,N", [(1, 32), (3, 512), (5, 544), (2, 2048), (7, 2080), (2, 8192), (1, 8224), (2, 32768),
                                 (2, 32800)])
def test_norm(M, N, out, dtype):
    log("norm M=%d N=%d out=%s dtype=%s" % (M, N, out, dtype))
    x, r, w = inputs(M, N, dtype, 1), inputs(M, N, dtype, 2, 3.0), inputs(1, N, dtype, 3)[0]
    y, scale, total = gr.rms_norm(x.cuda(), w.cuda(), r.cuda(), out_format=out)
    torch.cuda.synchronize()
    s, ref = norm_ref(x, r, w, 1e-6)
    assert torch.equal(total.cpu(), s)
    if out == "same":
        mx_ref.check16(y.cpu(), ref, x.dtype, ref.abs() * NORM)
    else:
        mx_ref.check_mx(y.cpu(), scale.cpu(), ref, out, NORM)


@pytest.mark.parametrize("M,N", [(1, 1), (2, 7), (3, 9), (2, 1501), (2, 4097), (1, 40001)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_odd_widths_and_pitches(M, N, residual):
    log("norm odd M=%d N=%d residual=%s" % (M, N, residual))
    x, r = inputs(M, N, "f16", 4), inputs(M, N, "f16", 5)
    _, vx = padded(x, N + 3, 1)
    _, vr = padded(r, N + 5, 3)
    by, vy = padded(torch.zeros_like(x), N + 2, 1)
    before = by.clone()
    y, scale, total = gr.rms_norm(vx, None, vr if residual else None, out_format="same", out=vy)
    torch.cuda.synchronize()
    s, ref = norm_ref(x, r if residual else None, None, 1e-6)
    assert scale is None and (total is None) == (not residual)
    mx_ref.check16(vy.cpu(), ref, x.dtype, ref.abs() * NORM)
    vy.copy_(torch.zeros_like(x))
    assert torch.equal(by.view(torch.int16), before.view(torch.int16)), "padding was written"


@pytest.mark.parametrize("N", [96, 8256, 33024])
def test_norm_mx_pitches_and_in_place_sum(N):
    log("norm mx pitches N=%d" % N)
    M = 3
    x, r = inputs(M, N, "bf16", 6), inputs(M, N, "bf16", 7)
    _, vx = padded(x, N + 9, 5)
    _, vr = padded(r, N + 7, 1)
    bq = torch.full((M * (N + 5) + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    q = bq[3:3 + M * (N + 5)].view(M, N + 5)[:, :N].view(torch.float8_e4m3fn)
    be = torch.full((M, N // 32 + 3), 0x5A, dtype=torch.uint8, device="cuda")
    y, scale, total = gr.rms_norm(vx, None, vr, out=q, scale_out=be[:, 1:1 + N // 32], sum_out=vr)
    torch.cuda.synchronize()
    s, ref = norm_ref(x, r, None, 1e-6)
    assert torch.equal(vr.cpu(), s)
    mx_ref.check_mx(y.cpu(), scale.cpu(), ref, "mxfp8", NORM)
    assert bool((be[:, 0] == 0x5A).all()) and bool((be[:, N // 32 + 1:] == 0x5A).all())
    rows = bq[3:3 + M * (N + 5)].view(M, N + 5)
    assert bool((rows[:, N:] == 0x5A).all()) and bool((bq[:3] == 0x5A).all())


def test_norm_in_place_16():
    x = inputs(5, 1024, "bf16", 8)
    d = x.cuda()
    gr.rms_norm(d, out_format="same", out=d)
    torch.cuda.synchronize()
    _, ref = norm_ref(x, None, None, 1e-6)
    mx_ref.check16(d.cpu(), ref, x.dtype, ref.abs() * NORM)


def test_norm_zero_rows_and_not_finite():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    x[1, 5], x[2, 40], x[3] = float("inf"), float("nan"), 2.0
    y, scale, _ = gr.rms_norm(x.cuda(), out_format="mxfp8")
    same, _, _ = gr.rms_norm(x.cuda(), out_format="same")
    torch.cuda.synchronize()
    y, scale, same = y.cpu().float(), scale.cpu(), same.cpu().float()
    assert bool((y[0] == 0).all()) and scale[0].tolist() == [0, 0] and bool((same[0] == 0).all())
    # inf * 0 and NaN: not finite where the value is, the rest of the row is 0 (inf) or NaN
    assert scale[1].tolist()[0] == 255 and scale[2].tolist() == [255, 255]
    assert bool(same[1, 5].isnan()) and bool(same[2].isnan().all())
    # 2 / sqrt(4 + eps) is just below 1: exponent -1, and 511.99 held to 448
    assert scale[3].tolist() == [127 - 9, 127 - 9] and bool((y[3] == 448).all())


# ---- quantisation and gated activation ------------------------------------------------

def every_value(dtype, top):
    """Rows of 32 with every non-negative finite 16-bit pattern up to `top` and its negative, next to blocks' largest
    value `top` itself, so the scale is fixed."""
    bits = torch.arange(0, 1 << 15, dtype=torch.int32).to(torch.int16)
    v = bits.view(mx_ref.TYPES[dtype]).float()
    v = v[v <= top]
    v = torch.cat((v, -v, torch.zeros(-2 * len(v) % 31)))
    rows = v.reshape(-1, 31)
    return torch.cat((torch.full((len(rows), 1), top), rows), 1).to(mx_ref.TYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt,top", [("mxfp8", 256.0), ("mxfp8", 508.0), ("mxfp4", 4.0), ("mxfp4", 7.5),
                                     ("mxfp4", 0.03125), ("mxfp8", 1.0)])
def test_quantise_every_value(fmt, top, dtype):
    """Bit-exact: one scaling by a power of two and one rounding."""
    x = every_value(dtype, top)
    log("quantise every value fmt=%s top=%g dtype=%s rows=%d" % (fmt, top, dtype, len(x)))
    y, scale = gr.mx_quantize(x.cuda(), fmt)
    torch.cuda.synchronize()
    q, e = mx_ref.quantise(x.double(), fmt)
    assert torch.equal(scale.cpu().int() - 127, e)
    assert torch.equal(mx_ref.elements(y.cpu(), fmt), q)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_quantise_extremes(fmt):
    """The ends of the exponent range, zeros, infinities, NaN, by block."""
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    x[0, :32] = torch.finfo(torch.bfloat16).max
    x[1, 3] = 2.0 ** -133  # the smallest subnormal
    x[2, 0], x[2, 1] = 2.0 ** -120, -(2.0 ** -126)
    x[3, 33] = float("-inf")
    x[4, 31] = float("nan")
    x[5] = -0.0
    x[6] = torch.tensor([1.0, -1.0] * 32)
    y, scale = gr.mx_quantize(x.cuda(), fmt)
    torch.cuda.synchronize()
    y, scale = mx_ref.elements(y.cpu(), fmt), scale.cpu()
    ok = torch.ones(8, 2, dtype=torch.bool)
    ok[3, 1] = ok[4, 0] = False
    assert bool((scale[~ok] == 255).all()) and bool((y.reshape(8, 2, 32)[~ok] == 0).all())
    q, e = mx_ref.quantise(torch.where(ok.repeat_interleave(32, 1), x.double(), 0.0), fmt)
    assert torch.equal((scale.int() - 127)[ok], e[ok])
    assert torch.equal(y.reshape(8, 2, 32)[ok], q.reshape(8, 2, 32)[ok])


@pytest.mark.parametrize("M,N", [(1, 32), (3, 4096), (5, 4128), (70, 160), (1, 65536)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "tanh", "sigmoid", "relu"])
@pytest.mark.parametrize("out", ["mxfp8", "mxfp4", "same"])
def test_gated(M, N, act, out):
    """The activations' fp32 forms are within a few ulp: 16 roundings with the product."""
    dtype = "bf16" if (M + N) % 3 else "f16"
    log("gated M=%d N=%d act=%s out=%s dtype=%s" % (M, N, act, out, dtype))
    g, u = inputs(M, N, dtype, 9, 3.0), inputs(M, N, dtype, 10)
    both = torch.cat((g, u), 1).cuda()  # the halves of one product
    y, scale = gr.gated_act(both[:, :N], both[:, N:], act, out)
    torch.cuda.synchronize()
    ref = mx_ref.act(g.double(), act) * u.double()
    # GELU's argument is rounded before the tail erfc(z) ~ exp(-z^2): z^2 more roundings
    extra = 16 * U + (2 * U * g.double().square().max().item() if act in ("gelu", "gelu_tanh") else 0)
    if out == "same":
        mx_ref.check16(y.cpu(), ref, g.dtype, ref.abs() * extra + 2.0 ** -126)
    else:
        mx_ref.check_mx(y.cpu(), scale.cpu(), ref, out, extra)


def test_gated_odd_width_in_place():
    g, u = inputs(6, 77, "f16", 11), inputs(6, 77, "f16", 12)
    bg, vg = padded(g, 83, 1)
    before = bg.clone()
    _, vu = padded(u, 79, 3)
    y, scale = gr.gated_act(vg, vu, "silu", "same", out=vg)
    torch.cuda.synchronize()
    ref = mx_ref.act(g.double(), "silu") * u.double()
    assert scale is None
    mx_ref.check16(vg.cpu(), ref, g.dtype, ref.abs() * 16 * U)
    vg.copy_(g)
    assert torch.equal(bg.view(torch.int16), before.view(torch.int16)), "padding was written"


def test_gated_infinities():
    g = torch.zeros(1, 32, dtype=torch.float16)
    g[0, :6] = torch.tensor([float("inf"), 60000.0, -60000.0, -100.0, -88.0, -0.0])
    for act, want in (("silu", [float("inf"), 60000.0, 0, 0, 0, 0]), ("sigmoid", [1, 1, 0, 0, 0, 0.5]),
                      ("gelu_tanh", [float("inf"), 60000.0, 0, 0, 0, 0]), ("tanh", [1, 1, -1, -1, -1, 0])):
        y, _ = gr.gated_act(g.cuda(), None, act, "same")
        assert y.cpu()[0, :6].float().tolist() == torch.tensor(want).half().float().tolist(), act


# ---- 16-bit activations, MX fp4 weights --------------------------------------------------

def weights(shape, K, seed, low=118, high=122):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(0, 256, (*shape, K // 2), generator=g, dtype=torch.uint8),
            torch.randint(low, high, (*shape, K // 32), generator=g, dtype=torch.uint8))


def check_linear(M, N, K, dtype, act="none", bias=False, low=118, high=122, seed=20):
    log("linear M=%d N=%d K=%d dtype=%s act=%s bias=%s scales=%d..%d" % (M, N, K, dtype, act, bias, low, high - 1))
    x = inputs(M, K, dtype, seed)
    w, s = weights((N,), K, seed + 1, low, high)
    b = inputs(1, N, dtype, seed + 2)[0] if bias else None
    out = gr.linear_mxfp4(x.cuda(), w.cuda(), s.cuda(), b.cuda() if bias else None, act)
    torch.cuda.synchronize()
    ref, mag = mx_ref.linear(x, w, s, b, act)
    mx_ref.check16(out.cpu(), ref, x.dtype, 1.2 * mag * mx_ref.sum_bound(K) + 8 * U * ref.abs())


@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 16, 64), (3, 17, 96), (2, 33, 128), (16, 40, 160), (17, 31, 192),
                                   (1, 64, 1024), (5, 100, 2080), (31, 48, 416), (33, 65, 288), (64, 80, 544),
                                   (65, 32, 256), (130, 50, 1056), (16, 64, 4096)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear(M, N, K, dtype):
    check_linear(M, N, K, dtype)


@pytest.mark.parametrize("M,N,K", [(3, 20, 8736), (16, 50, 16384), (17, 33, 4640), (32, 1040, 8192), (33, 65, 2080),
                                   (64, 100, 6176), (64, 640, 2048), (70, 17, 4128)])
@pytest.mark.parametrize("workspace", ["auto", None])
def test_linear_long_k(M, N, K, workspace):
    """A K that one workgroup cannot hold: several workgroups with a workspace, several passes without."""
    dtype = "bf16" if M % 2 else "f16"
    log("linear long k M=%d N=%d K=%d dtype=%s workspace=%s" % (M, N, K, dtype, workspace))
    x = inputs(M, K, dtype, 25)
    w, s = weights((N,), K, 26)
    b = inputs(1, N, dtype, 27)[0]
    out = gr.linear_mxfp4(x.cuda(), w.cuda(), s.cuda(), b.cuda(), "silu", workspace=workspace)
    torch.cuda.synchronize()
    ref, mag = mx_ref.linear(x, w, s, b, "silu")
    mx_ref.check16(out.cpu(), ref, x.dtype, 1.2 * mag * mx_ref.sum_bound(K) + 8 * U * ref.abs())


def test_linear_wide_scales_f16():
    """fp16 rows whose scales differ by more than the conversion holds (2^13): the block by block form, beside
    rows that do not."""
    M, N, K = 7, 48, 1024
    x = inputs(M, K, "f16", 28)
    w, s = weights((N,), K, 29)
    g = torch.Generator().manual_seed(30)
    s[5] = torch.randint(96, 126, (K // 32,), generator=g, dtype=torch.uint8)
    s[20, 7] = 0
    s[21, 0] = 0
    s[40] = torch.randint(60, 80, (K // 32,), generator=g, dtype=torch.uint8)
    out = gr.linear_mxfp4(x.cuda(), w.cuda(), s.cuda())
    torch.cuda.synchronize()
    ref, mag = mx_ref.linear(x, w, s)
    mx_ref.check16(out.cpu(), ref, x.dtype, mag * mx_ref.sum_bound(K))


@pytest.mark.parametrize("M,N,K", [(1, 16400, 64), (17, 16390, 32), (40, 16385, 128), (16, 20000, 256)])
def test_linear_many_columns(M, N, K):
    check_linear(M, N, K, "bf16")


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "sigmoid", "tanh"])
def test_linear_epilogue(act):
    check_linear(9, 52, 320, "f16", act, True)


@pytest.mark.parametrize("low,high,scale", [(0, 3, 2.0 ** 100), (250, 255, 2.0 ** -126)])
def test_linear_scale_extremes(low, high, scale):
    """Every scale code to the ends of E8M0 is exact (bfloat16 has the range to show it)."""
    x = inputs(4, 256, "bf16", 30, scale)
    w, s = weights((40,), 256, 31, low, high)
    out = gr.linear_mxfp4(x.cuda(), w.cuda(), s.cuda())
    torch.cuda.synchronize()
    ref, mag = mx_ref.linear(x, w, s)
    mx_ref.check16(out.cpu(), ref, x.dtype, mag * mx_ref.sum_bound(256) + 256 * 2.0 ** -126)


def test_linear_nan_scale_and_row():
    """Scale code 255 makes its weight row's column NaN, a NaN or infinity of x its own row, and nothing else."""
    x = inputs(20, 160, "f16", 32)
    w, s = weights((24,), 160, 33)
    w[:, :] = w | 0x11  # no zero weights: 0 * inf would hide among the NaN
    s[5, 4], s[7, 0] = 255, 255
    x[3, 150] = float("nan")
    x[11, 2] = float("inf")
    out = gr.linear_mxfp4(x.cuda(), w.cuda(), s.cuda()).cpu()
    bad = torch.zeros(20, 24, dtype=torch.bool)
    bad[:, 5] = bad[:, 7] = True
    bad[3] = bad[11] = True
    assert torch.equal(~out.isfinite(), bad)
    assert bool(out[:, [5, 7]].isnan().all()) and bool(out[3].isnan().all())


def test_linear_pitches_and_stream():
    """Padded rows at odd addresses on a stream of their own; nothing outside C is written."""
    M, N, K = 19, 45, 288
    x = inputs(M, K, "bf16", 34)
    w, s = weights((N,), K, 35)
    _, vx = padded(x, K + 3, 1)
    _, vw = padded(w, K // 2 + 5, 3)
    _, vs = padded(s, K // 32 + 1, 1, fill=0xFF)
    bc, vc = padded(torch.zeros(M, N, dtype=torch.bfloat16), N + 3, 1)
    before = bc.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    gr.linear_mxfp4(vx, vw, vs, out=vc, stream=side)
    side.synchronize()
    ref, mag = mx_ref.linear(x, w, s)
    mx_ref.check16(vc.cpu(), ref, x.dtype, mag * mx_ref.sum_bound(K))
    vc.copy_(torch.zeros(M, N, dtype=torch.bfloat16))
    assert torch.equal(bc.view(torch.int16), before.view(torch.int16)), "padding was written"


def test_linear_empty_k():
    b = inputs(1, 9, "f16", 36)[0]
    x = torch.zeros(3, 0, dtype=torch.float16, device="cuda")
    w = torch.zeros(9, 0, dtype=torch.uint8, device="cuda")
    out = gr.linear_mxfp4(x, w, w, b.cuda(), "relu")
    assert torch.equal(out.cpu(), b.clamp(min=0).expand(3, 9))


def test_quantised_product():
    """mx_quantize feeds gemm_mxfp4: the product of the quantised values."""
    x, w = inputs(37, 256, "bf16", 37), inputs(48, 256, "bf16", 38)
    (qa, sa), (qb, sb) = gr.mx_quantize(x.cuda(), "mxfp4"), gr.mx_quantize(w.cuda(), "mxfp4")
    out = gr.gemm_mxfp4(qa, sa, qb, sb, act="none", out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    a, b = mx_ref.weight(qa.cpu(), sa.cpu()), mx_ref.weight(qb.cpu(), sb.cpu())
    # the matrix cores' own sums: 2^-16 of the absolute products, as the MX fp4 tests allow
    mx_ref.check16(out.cpu(), a @ b.T, torch.bfloat16, (a.abs() @ b.abs().T) * 2.0 ** -16)


def check_fp4(M, N, K, dtype="bf16", act="none", bias=False, low=118, high=124, seed=90, **kw):
    log("fp4 x fp4 M=%d N=%d K=%d dtype=%s act=%s bias=%s scales=%d..%d" % (M, N, K, dtype, act, bias, low, high - 1))
    (qa, sa), (qb, sb) = weights((M,), K, seed, low, high), weights((N,), K, seed + 1, 250 - high, 250 - low)
    b = inputs(1, N, dtype, seed + 2)[0] if bias else None
    out = gr.gemm_mxfp4(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), b.cuda() if bias else None, act,
                        mx_ref.TYPES[dtype], **kw)
    torch.cuda.synchronize()
    a, w = mx_ref.weight(qa, sa), mx_ref.weight(qb, sb)
    v, mag = a @ w.T, a.abs() @ w.abs().T
    if bias:
        v, mag = v + b.double(), mag + b.double().abs()
    # the matrix cores' own sums, as the MX fp4 tests allow; 1.2: the steepest activation
    ref = mx_ref.act(v, act)
    mx_ref.check16(out.cpu(), ref, mx_ref.TYPES[dtype], 1.2 * mag * (2.0 ** -16 + mx_ref.sum_bound(K)) + 8 * U * ref.abs())


@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (2, 17, 64), (16, 16, 96), (5, 40, 128), (17, 33, 160), (64, 48, 480),
                                   (65, 50, 512), (100, 130, 1056), (1, 1000, 2080), (200, 100, 4096), (3, 40, 4128),
                                   (33, 70, 8224), (130, 600, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_fp4_product(M, N, K, dtype):
    check_fp4(M, N, K, dtype)


@pytest.mark.parametrize("strips", [1, 2, 3, 4, 5, 6, 7, 8, 9, 16, 31])
@pytest.mark.parametrize("M,N", [(130, 200), (128, 256)])
def test_fp4_product_tiles(M, N, strips):
    """The 128 x 128 tiles: whole ones and edges, every remainder of their ring of strips."""
    check_fp4(M, N, 128 * strips, "f16" if strips % 2 else "bf16", path=gr.GR_PATH_TILE)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "sigmoid", "tanh"])
def test_fp4_product_epilogue(act):
    check_fp4(21, 37, 352, "f16", act, True)
    check_fp4(3, 70, 4160, "bf16", act, True)


def test_fp4_product_scale_extremes():
    check_fp4(5, 20, 256, low=0, high=2)
    check_fp4(18, 20, 256, low=248, high=250)


def test_fp4_product_nan_scales():
    """Scale code 255 on either side makes its row or column NaN and nothing else."""
    (qa, sa), (qb, sb) = weights((20,), 160, 93), weights((24,), 160, 94)
    sa[3, 4] = sb[5, 0] = 255
    out = gr.gemm_mxfp4(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), act="none").cpu()
    bad = torch.zeros(20, 24, dtype=torch.bool)
    bad[3] = bad[:, 5] = True
    assert torch.equal(out.isnan(), bad)


def test_fp4_product_pitches():
    """Padded rows at odd addresses, nothing outside the output written."""
    M, N, K = 19, 45, 288
    (qa, sa), (qb, sb) = weights((M,), K, 95), weights((N,), K, 96)
    views = [padded(t, t.shape[1] + p, o, fill=0xFF)[1] for t, p, o in ((qa, 5, 3), (sa, 1, 1), (qb, 3, 1), (sb, 2, 3))]
    bc, vc = padded(torch.zeros(M, N, dtype=torch.bfloat16), N + 3, 1)
    before = bc.clone()
    gr.gemm_mxfp4(*views, act="none", out=vc)
    torch.cuda.synchronize()
    a, w = mx_ref.weight(qa, sa), mx_ref.weight(qb, sb)
    mx_ref.check16(vc.cpu(), a @ w.T, torch.bfloat16, (a.abs() @ w.abs().T) * (2.0 ** -16 + mx_ref.sum_bound(K)))
    vc.copy_(torch.zeros(M, N, dtype=torch.bfloat16))
    assert torch.equal(bc.view(torch.int16), before.view(torch.int16)), "padding was written"


# ---- mixture of experts -------------------------------------------------------------------

@pytest.mark.parametrize("T,H,E,k", [(1, 64, 4, 1), (3, 96, 8, 8), (16, 100, 17, 3), (17, 1000, 64, 8), (5, 33, 65, 4),
                                     (2, 256, 256, 8), (4, 64, 1000, 32), (2, 4096, 128, 4), (1, 1, 2, 1)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, H, E, k, renorm):
    log("route T=%d H=%d E=%d k=%d renorm=%s" % (T, H, E, k, renorm))
    dtype = "bf16" if T % 2 else "f16"
    x, w = inputs(T, H, dtype, 40), inputs(E, H, dtype, 41, 2 * H ** -0.5)
    b = torch.randn(E, generator=torch.Generator().manual_seed(42)) if renorm else None
    ids, weights_ = gr.moe_route(x.cuda(), w.cuda(), k, b.cuda() if renorm else None, renorm)
    torch.cuda.synchronize()
    ids, weights_ = ids.cpu().long(), weights_.cpu().double()
    logits = x.double() @ w.double().T + (b.double() if renorm else 0)
    mag = x.double().abs() @ w.double().abs().T + (b.double().abs() if renorm else 0)
    off = (mag * mx_ref.sum_bound(H)).max().item()
    best = logits.sort(-1, descending=True).values[:, :k]
    assert bool((logits.gather(1, ids) - best).abs().max() <= 2 * off)
    assert all(len(set(r)) == k for r in ids.tolist())
    top = logits.gather(1, ids)
    e = torch.exp(top - logits.amax(-1, keepdim=True))
    total = e.sum(-1, keepdim=True) if renorm else torch.exp(logits - logits.amax(-1, keepdim=True)).sum(-1, keepdim=True)
    assert bool(((weights_ - e / total).abs() <= (e / total) * (4 * off + 64 * U)).all())


@pytest.mark.parametrize("T,H,E,k", [(1, 4096, 64, 8), (5, 2080, 40, 3), (33, 1500, 129, 6), (2, 700, 1000, 20),
                                     (512, 1100, 64, 2)])
def test_route_workspace(T, H, E, k):
    """With a workspace (two kernels) and without: both are the topk of logits within the sums' bounds."""
    x, w = inputs(T, H, "bf16", 43), inputs(E, H, "bf16", 44, 2 * H ** -0.5)
    st, size = gr.moe_route_workspace_size(T, H, E)
    assert st == gr.GR_OK and size > 0
    logits = x.double() @ w.double().T
    off = (x.double().abs() @ w.double().abs().T * mx_ref.sum_bound(H)).max().item()
    best = logits.sort(-1, descending=True).values[:, :k]
    for workspace in ("auto", None):
        log("route workspace T=%d H=%d E=%d k=%d %s" % (T, H, E, k, workspace))
        ids, p = gr.moe_route(x.cuda(), w.cuda(), k, workspace=workspace)
        torch.cuda.synchronize()
        ids, p = ids.cpu().long(), p.cpu().double()
        top = logits.gather(1, ids)
        assert bool((top - best).abs().max() <= 2 * off) and all(len(set(r)) == k for r in ids.tolist())
        ref = torch.softmax(top, -1)
        assert bool(((p - ref).abs() <= ref * (4 * off + 64 * U)).all())


def test_route_ties_and_not_finite():
    """Equal logits (exact whole numbers) go to the lower index; NaN is chosen first; -inf rows still give distinct ids."""
    x = torch.ones(3, 32, dtype=torch.bfloat16)
    w = torch.zeros(70, 32, dtype=torch.bfloat16)
    w[:, 0] = torch.tensor([float(v) for v in ([3, 1, 3, 2] * 18)[:70]])
    ids, weights_ = gr.moe_route(x.cuda(), w.cuda(), 20)
    assert ids.cpu()[0].tolist() == [e for e in range(70) if w[e, 0] == 3][:20]
    assert bool((weights_.cpu() == torch.tensor(1.0) / 20).all())
    bias = torch.zeros(70)
    bias[69] = float("nan")
    ids, weights_ = gr.moe_route(x.cuda(), w.cuda(), 2, bias.cuda())
    assert ids.cpu()[1].tolist() == [69, 0] and bool(weights_.cpu().isnan().all())
    ids, weights_ = gr.moe_route(x.cuda(), w.cuda(), 3, torch.full((70,), float("-inf")).cuda())
    assert ids.cpu()[2].tolist() == [0, 1, 2] and bool(weights_.cpu().isnan().all())


def check_moe(T, H, I, E, k, dtype, act="silu", bias=False, seed=50, ids=None):
    log("moe T=%d H=%d I=%d E=%d k=%d dtype=%s act=%s bias=%s" % (T, H, I, E, k, dtype, act, bias))
    g = torch.Generator().manual_seed(seed)
    x = inputs(T, H, dtype, seed + 1)
    (w13, s13), (w2, s2) = weights((E, 2 * I), H, seed + 2), weights((E, H), I, seed + 3)
    if ids is None:
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    p = torch.rand(T, k, generator=g)
    b13 = inputs(E, 2 * I, dtype, seed + 4) if bias else None
    b2 = inputs(E, H, dtype, seed + 5) if bias else None
    dev = [None if t is None else t.cuda() for t in (x, ids, p, w13, s13, w2, s2, b13, b2)]
    out = gr.moe_mxfp4(*dev, act=act)
    torch.cuda.synchronize()
    ref, bound = mx_ref.moe(x, ids, p, w13, s13, w2, s2, b13, b2, act)
    mx_ref.check16(out.cpu(), ref, x.dtype, bound)
    again = gr.moe_mxfp4(*dev, act=act)
    assert torch.equal(again.cpu().view(torch.int16), out.cpu().view(torch.int16)), "the result depends on timing"
    return out


@pytest.mark.parametrize("T,H,I,E,k", [(1, 32, 32, 1, 1), (1, 64, 96, 4, 2), (2, 160, 64, 8, 8), (7, 256, 160, 5, 3),
                                       (16, 128, 128, 3, 2), (17, 96, 288, 4, 2), (40, 64, 64, 2, 2),
                                       (64, 128, 96, 6, 4), (65, 64, 128, 7, 2), (130, 32, 64, 9, 3),
                                       (3, 512, 1024, 64, 6), (5, 64, 64, 600, 4), (2, 64, 2080, 3, 3), (1, 96, 1056, 9, 4),
                                       (12, 4128, 32, 3, 2), (20, 8224, 64, 2, 1), (18, 32, 4160, 2, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_moe(T, H, I, E, k, dtype):
    check_moe(T, H, I, E, k, dtype, bias=(T % 2 == 0))


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh"])
def test_moe_activations(act):
    check_moe(6, 96, 64, 5, 2, "bf16", act, True)


def test_moe_absent_and_repeated_experts():
    """Ids outside [0, E) are passed over, a token without experts gives zeros, a repeated expert counts twice."""
    ids = torch.tensor([[-1, 7, 3], [2, 2, 2], [-5, 9, 1 << 30], [0, -1, 0], [4, 4, 1]], dtype=torch.int32)
    out = check_moe(5, 64, 96, 5, 3, "bf16", bias=True, ids=ids)
    assert bool((out[2] == 0).all())
    out = check_moe(5, 64, 96, 5, 3, "f16", ids=torch.full((5, 3), -1, dtype=torch.int32))
    assert bool((out == 0).all())


def test_moe_nan_reaches_only_its_tokens():
    """A NaN scale of one expert, and an infinity in one token, stay with the tokens that use them."""
    T, H, I, E = 18, 128, 64, 4
    x = inputs(T, H, "bf16", 60)
    (w13, s13), (w2, s2) = weights((E, 2 * I), H, 61), weights((E, H), I, 62)
    s2[1, 3, 0] = 255
    s13[2, 5, 1] = 255
    x[4, 9] = float("nan")
    ids = torch.tensor([[t % 4] for t in range(T)], dtype=torch.int32)
    p = torch.ones(T, 1)
    out = gr.moe_mxfp4(*(t.cuda() for t in (x, ids, p, w13, s13, w2, s2))).cpu()
    for t in range(T):
        bad = out[t].isnan()
        want = torch.zeros(H, dtype=torch.bool)
        if t % 4 == 1:
            want[3] = True
        if t % 4 == 2 or t == 4:
            want[:] = True
        assert torch.equal(bad, want), t


def test_moe_workspace_contents_do_not_matter():
    T, H, I, E, k = 9, 64, 96, 6, 2
    x = inputs(T, H, "f16", 70)
    (w13, s13), (w2, s2) = weights((E, 2 * I), H, 71), weights((E, H), I, 72)
    ids, p = torch.randint(0, E, (T, k), dtype=torch.int32), torch.rand(T, k)
    dev = [t.cuda() for t in (x, ids, p, w13, s13, w2, s2)]
    st, size = gr.moe_w4_workspace_size(T, H, I, E, k)
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    a = gr.moe_mxfp4(*dev, workspace=ws[:size])
    b = gr.moe_mxfp4(*dev)
    assert torch.equal(a.cpu(), b.cpu()) and bool((ws[size:] == 0xFF).all())
    with pytest.raises(gr.GemmReluError):
        gr.moe_mxfp4(*dev, workspace=ws[:size - 256])


def test_block_in_a_graph():
    """The block as a decoding step runs it, captured once and replayed: equal to the eager result every time."""
    T, H, I, E, k = 4, 256, 128, 8, 2
    x, r = inputs(T, H, "bf16", 80).cuda(), inputs(T, H, "bf16", 81).cuda()
    router = inputs(E, H, "bf16", 82, 2 * H ** -0.5).cuda()
    (w13, s13), (w2, s2), (wo, so) = weights((E, 2 * I), H, 83), weights((E, H), I, 84), weights((96,), H, 85)
    dev = [t.cuda() for t in (w13, s13, w2, s2, wo, so)]

    def step():
        y, _, total = gr.rms_norm(x, None, r, out_format="same")
        ids, p = gr.moe_route(y, router, k)
        z = gr.moe_mxfp4(y, ids, p, *dev[:4])
        n, _, _ = gr.rms_norm(z, None, total, out_format="same")
        return gr.linear_mxfp4(n, dev[4], dev[5], act="gelu")

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(4):
        x.copy_(inputs(T, H, "bf16", 90 + i))
        want = step().cpu()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured.cpu().view(torch.int16), want.view(torch.int16)), i


# ---- the blocks --------------------------------------------------------------------------

def block_inputs(T, H, I, E, seed):
    x, r, n = inputs(T, H, "bf16", seed), inputs(T, H, "bf16", seed + 1), (1 + inputs(1, H, "bf16", seed + 2, 0.1)[0])
    return x, r, n.bfloat16(), inputs(2 * I * max(E, 1), H, "bf16", seed + 3, 0.05), inputs(H * max(E, 1), I, "bf16",
                                                                                            seed + 4, 0.05)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_dense_blocks(T):
    """Each step's rounding to bfloat16 (or MX fp4) is repeated in the plain form, so that only the sums differ: the
    products' inputs agree but for values next to a rounding border, which a comparison of norms allows for."""
    from dense_gemm_epilogue_tiled_amd import feed_forward as ff
    H, I = 256, 192
    x, r, n, w13, w2 = block_inputs(T, H, I, 0, 100)
    q13, q2 = ff.quantize_weight(w13.cuda()), ff.quantize_weight(w2.cuda())
    a, b = mx_ref.weight(q13[0].cpu(), q13[1].cpu()), mx_ref.weight(q2[0].cpu(), q2[1].cpu())
    total, h = norm_ref(x, r, n, 1e-6)
    for fp4 in (False, True):
        out, got_total = (ff.dense_block_fp4 if fp4 else ff.dense_block)(x.cuda(), r.cuda(), n.cuda(), q13, q2)
        assert torch.equal(got_total.cpu(), total)

        def rounded(v):
            if not fp4:
                return v.bfloat16().double()
            q, e = mx_ref.quantise(v, "mxfp4")
            return q * torch.pow(2.0, e.double()).repeat_interleave(32, -1)

        both = (rounded(h) @ a.T).bfloat16().double()
        ref = rounded(mx_ref.act(both[:, :I], "silu") * both[:, I:]) @ b.T
        err = (out.cpu().double() - ref).norm() / ref.norm()
        # half steps of bfloat16 in the output and, where a border was crossed, in the inputs; an fp4 element
        # that crosses one is off by half of itself, which few do
        assert err < (2.0 ** -8 * 2 if not fp4 else 0.05), (fp4, float(err))


@pytest.mark.parametrize("T", [1, 6, 40])
def test_moe_block(T):
    from dense_gemm_epilogue_tiled_amd import feed_forward as ff
    H, I, E, k = 256, 128, 8, 2
    x, r, n, w13, w2 = block_inputs(T, H, I, E, 110)
    router = inputs(E, H, "bf16", 120, 2 * H ** -0.5)
    q13, q2 = ff.quantize_weight(w13.view(E, 2 * I, H).cuda()), ff.quantize_weight(w2.view(E, H, I).cuda())
    out, got_total = ff.moe_block(x.cuda(), r.cuda(), n.cuda(), router.cuda(), k, q13, q2)
    h, _, _ = gr.rms_norm(x.cuda(), n.cuda(), r.cuda(), out_format="same")
    ids, p = gr.moe_route(h, router.cuda(), k)
    total, _ = norm_ref(x, r, n, 1e-6)
    assert torch.equal(got_total.cpu(), total)
    ref, bound = mx_ref.moe(h.cpu(), ids.cpu(), p.cpu(), *(t.cpu() for t in (*q13, *q2)), None, None, "silu")
    mx_ref.check16(out.cpu(), ref, torch.bfloat16, bound)


# ---- what all of them share ------------------------------------------------------------------

def test_empty_tensors():
    """No rows, no columns, no tokens: empty results, nothing launched on them."""
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    w, s = torch.zeros(8, 32, dtype=torch.uint8, device="cuda"), torch.zeros(8, 2, dtype=torch.uint8, device="cuda")
    y, scale, total = gr.rms_norm(x, residual=x)
    assert y.shape == (0, 64) and scale.shape == (0, 2) and total.shape == (0, 64)
    assert gr.rms_norm(x[:, :0], out_format="same")[0].shape == (0, 0)
    y, scale = gr.gated_act(x, x)
    assert y.shape == (0, 64) and scale.shape == (0, 2)
    assert gr.linear_mxfp4(x, w, s).shape == (0, 8)
    one = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    assert gr.linear_mxfp4(one, w[:0], s[:0]).shape == (3, 0)
    assert gr.gemm_mxfp4(w[:0], s[:0], w, s).shape == (0, 8) and gr.gemm_mxfp4(w, s, w[:0], s[:0]).shape == (8, 0)
    ids, p = gr.moe_route(x, one, 2)
    assert ids.shape == p.shape == (0, 2)
    w13, s13 = torch.zeros(2, 64, 32, dtype=torch.uint8, device="cuda"), torch.zeros(2, 64, 2, dtype=torch.uint8,
                                                                                  device="cuda")
    w2, s2 = torch.zeros(2, 64, 16, dtype=torch.uint8, device="cuda"), torch.zeros(2, 64, 1, dtype=torch.uint8,
                                                                                 device="cuda")
    assert gr.moe_mxfp4(x, ids, p, w13, s13, w2, s2).shape == (0, 64)
    torch.cuda.synchronize()


def test_empty_intermediate():
    """Experts without an intermediate dimension leave their biases."""
    x = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(2, 0, 32, dtype=torch.uint8, device="cuda"), torch.zeros(2, 0, 2, dtype=torch.uint8, device="cuda")
    w2, s2 = torch.zeros(2, 64, 0, dtype=torch.uint8, device="cuda"), torch.zeros(2, 64, 0, dtype=torch.uint8,
                                                                                device="cuda")
    b2 = inputs(2, 64, "bf16", 130)
    ids = torch.tensor([[0], [1], [-1]], dtype=torch.int32, device="cuda")
    out = gr.moe_mxfp4(x, ids, torch.ones(3, 1, device="cuda"), *none, w2, s2, b2=b2.cuda()).cpu()
    assert torch.equal(out[:2], b2) and bool((out[2] == 0).all())


def test_streams():
    """On a stream given as an object or as a handle, new tensors included: the same bits as on the current one."""
    x, r = inputs(5, 512, "bf16", 140).cuda(), inputs(5, 512, "bf16", 141).cuda()
    (w, s), (w13, s13), (w2, s2) = weights((96,), 512, 142), weights((4, 128), 512, 143), weights((4, 512), 64, 144)
    dev = [t.cuda() for t in (w, s, w13, s13, w2, s2)]
    router = inputs(4, 512, "bf16", 145).cuda()

    def step(**kw):
        y, _, total = gr.rms_norm(x, None, r, out_format="same", **kw)
        ids, p = gr.moe_route(y, router, 2, **kw)
        z = gr.moe_mxfp4(y, ids, p, *dev[2:], **kw)
        q, scale = gr.mx_quantize(z, "mxfp4", **kw)
        g, _ = gr.gated_act(z, total, "silu", "same", **kw)
        return gr.linear_mxfp4(g, *dev[:2], **kw), gr.gemm_mxfp4(q, scale, *dev[:2], **kw)

    want = [t.cpu() for t in step()]
    torch.cuda.synchronize()
    for _ in range(3):
        side = torch.cuda.Stream()
        for stream in (side, side.cuda_stream):
            got = step(stream=stream)
            side.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a.cpu().view(torch.int16), b.view(torch.int16))


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 bytes apart, in the activations and over all rows of the weights."""
    pitch = (1 << 31) + 24
    buf = torch.empty(2 * pitch + 4096, dtype=torch.bfloat16, device="cuda")
    x = inputs(3, 512, "bf16", 150)
    vx = buf.as_strided((3, 512), (pitch, 1))
    vx.copy_(x)
    y, scale, _ = gr.rms_norm(vx)
    s, ref = norm_ref(x, None, None, 1e-6)
    mx_ref.check_mx(y.cpu(), scale.cpu(), ref, "mxfp8", NORM)
    y, scale = gr.mx_quantize(vx, "mxfp4")
    q, e = mx_ref.quantise(x.double(), "mxfp4")
    assert torch.equal(mx_ref.elements(y.cpu(), "mxfp4"), q) and torch.equal(scale.cpu().int() - 127, e)
    N, step = 300, 1 << 24
    w, ws = weights((N,), 512, 151)
    wide = buf.view(torch.uint8).as_strided((N, 256), (step, 1), 4096)
    wide.copy_(w)
    vx = inputs(3, 512, "bf16", 152).cuda()
    out = gr.linear_mxfp4(vx, wide, ws.cuda())
    ref, mag = mx_ref.linear(vx.cpu(), w, ws)
    mx_ref.check16(out.cpu(), ref, torch.bfloat16, mag * mx_ref.sum_bound(512))
    out = gr.gemm_mxfp4(*gr.mx_quantize(vx, "mxfp4"), wide, ws.cuda(), act="none", out_dtype=torch.bfloat16)
    q, e = mx_ref.quantise(vx.cpu().double(), "mxfp4")
    a, b = q * torch.pow(2.0, e.double()).repeat_interleave(32, -1), mx_ref.weight(w, ws)
    mx_ref.check16(out.cpu(), a @ b.T, torch.bfloat16, (a.abs() @ b.abs().T) * (2.0 ** -16 + mx_ref.sum_bound(512)))
