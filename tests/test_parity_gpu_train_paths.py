"""GPU tests of the training operators that name the kernel they are meant for: each runs a size that the operator gives to
that kernel, checks it against the plain fp64 forms (train_ref) with rows apart and odd addresses around, and then checks by
the names of the launched kernels that it was the one. A border that moves fails here, not silently elsewhere."""
import re

import pytest
import torch

import dense_gemm_epilogue_tiled_amd as gr
import train_ref
from gpu_util import log
from mx_ref import check16
from train_ref import TYPES, make

pytestmark = pytest.mark.gpu

ELEM = {"bf16": "gr::ElemBF16", "f16": "gr::ElemF16"}


def launched(call):
    """call's result and the names of the kernels that it launched, up to their arguments."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        out = call()
        torch.cuda.synchronize()
    names = [e.name for e in p.events() if e.device_type == torch.autograd.DeviceType.CUDA]
    return out, [re.sub(r"^void |\(anonymous namespace\)::|\(gr::ortho::FoldTo\)", "", n).split("(")[0] for n in names]


def check_launched(names, *wanted):
    if not names:
        pytest.skip("the results are right; no kernel names are recorded here")
    for w in wanted:
        assert any(w in n for n in names), (w, names)


def tile256(epilogue, ragged, kernel="tile3t"):
    return "gemm_relu_%s_kernel<%s, %s" % (kernel, "true" if ragged else "false", epilogue)


def tile128(epilogue, ragged):
    return "gemm_relu_tile128_kernel<%s, false, true, %s" % ("true" if ragged else "false", epilogue)


def stream(epilogue, waves, rows):
    return "gemm_relu_smallm_stream_kernel<64, %d, 2, 0, %s, false, %d, true, true>" % (waves, epilogue, rows // 16)


def own(name, dtype):
    return "gr::own::%s<%s>" % (name, ELEM[dtype])


def dev(t, pad=0, offset=0):
    """t on the GPU, its rows `pad` elements further apart and its first `offset` elements behind a 256-byte border, in a
    buffer of NaN."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + offset + 64,), float("nan"), dtype=t.dtype, device="cuda")
    v = torch.as_strided(buf, (rows, cols), (cols + pad, 1), offset)
    v.copy_(t)
    return v


class Guarded:
    """An output at an odd address whose rows are an odd number of elements apart, in a buffer of 77."""

    def __init__(self, rows, cols, dtype):
        self.buf = torch.full((rows + 2, cols + 5 + cols % 2), 77.0, dtype=dtype, device="cuda")
        self.view = self.buf[1:rows + 1, 1:cols + 1]

    def check(self):
        got = self.view.cpu()
        self.view.fill_(77.0)
        assert bool((self.buf == 77).all())
        return got


# ---- gated linear layer ----------------------------------------------------------------------

# M, I, H and the kernel. 256 x 256 tiles hold 128 columns, 128 x 128 tiles 64, streamed blocks 32
GATED = [(512, 8320, 320, lambda e: tile256(e, False)), (500, 8300, 192, lambda e: tile256(e, True)),
         (500, 8300, 90, lambda e: tile256(e, True)), (256, 2112, 320, lambda e: tile128(e, False)),
         (200, 2100, 96, lambda e: tile128(e, True)), (50, 6390, 96, lambda e: stream(e, 8, 64)),
         (64, 9001, 64, lambda e: stream(e, 4, 64)), (130, 4200, 1024, lambda e: stream(e, 4, 64)),
         (77, 700, 352, lambda e: stream(e, 8, 32))]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,I,H,kernel", GATED, ids=lambda v: str(v) if isinstance(v, int) else "")
def test_gated_linear_paths(M, I, H, kernel, dtype):
    log("gated path %dx%dx%d %s" % (M, I, H, dtype))
    x, w, b = make((M, H), dtype, 1), make((2 * I, H), dtype, 2, H ** -0.5), make((2 * I,), dtype, 3)
    out, gu = Guarded(M, I, TYPES[dtype]), Guarded(M, 2 * I, TYPES[dtype])
    xs, ws, bs = dev(x, 8 if H % 8 == 0 else 3), dev(w, 8 if H % 8 == 0 else 3), b.cuda()
    _, names = launched(lambda: gr.gated_linear(xs, ws, bs, act="silu", keep=True, out=out.view, gu_out=gu.view))
    ref, bound, ref_gu, bound_gu = train_ref.gated(x, w, b, "silu")
    check16(out.check(), ref, TYPES[dtype], bound)
    check16(gu.check(), ref_gu, TYPES[dtype], bound_gu)
    check_launched(names, kernel(own("Gated", dtype)))


# ---- gradients of linear layers ----------------------------------------------------------------

def bare(dtype, ragged):
    return tile256("Bare<%s>" % ELEM[dtype], ragged, "tile3")


def plain(kernel, *args):
    return lambda dtype: kernel(own("Plain", dtype), *args)


# M, N, K, padding of the weight's rows, the input's kernel (of dX, M x K, sums over N) and the weight's (of dW, N x K, sums
# over the tokens), None: another test's
LINEAR = [(8448, 64, 1024, 0, lambda d: bare(d, False), None), (8448, 320, 1024, 8, lambda d: bare(d, False), None),
          (8400, 128, 1000, 0, lambda d: bare(d, True), None), (8400, 320, 1003, 5, lambda d: bare(d, True), None),
          (33100, 64, 72, 0, lambda d: bare(d, True), None), (33025, 192, 256, 0, lambda d: bare(d, True), None),
          (200, 2816, 3328, 0, None, plain(tile256, False)), (300, 2700, 3301, 0, None, plain(tile256, True)),
          (1, 2700, 3300, 0, None, plain(tile256, True)), (4096, 100, 1024, 0, plain(tile128, False), None),
          (4100, 100, 1001, 0, plain(tile128, True), None), (100, 4001, 1000, 0, plain(stream, 8, 32), None),
          (300, 1001, 4100, 0, plain(stream, 4, 64), None)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,pad,input_kernel,weight_kernel", LINEAR, ids=lambda v: str(v) if isinstance(v, int) else "")
def test_linear_backward_paths(M, N, K, pad, input_kernel, weight_kernel, dtype):
    log("linear backward path %dx%dx%d %s" % (M, N, K, dtype))
    dy, x, w = make((M, N), dtype, 11), make((M, K), dtype, 12), make((N, K), dtype, 13, K ** -0.5)
    dx, dw = Guarded(M, K, TYPES[dtype]), Guarded(N, K, TYPES[dtype])
    dys, xs, ws = dy.cuda(), dev(x, 1, 3), dev(w, pad)
    got, names = launched(lambda: gr.linear_backward(dys, xs, ws, bias=True, dx_out=dx.view, dw_out=dw.view))
    refs, bounds = train_ref.linear_backward(dy, x, w)
    for g, r, b in zip((dx.check(), dw.check(), got[2].cpu()), refs, bounds):
        check16(g, r, TYPES[dtype], b)
    check_launched(names, *[k(dtype) for k in (input_kernel, weight_kernel) if k])


# M, I, H and the kernels of dX (M x H, sums over 2I) and dW13 (2I x H, sums over the tokens)
GATED_BWD = [(8448, 32, 1024, lambda d: bare(d, False), None), (8400, 96, 1000, lambda d: bare(d, True), None),
             (200, 1408, 3328, None, plain(tile256, False)), (130, 1350, 3301, None, plain(tile256, True))]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,I,H,input_kernel,weight_kernel", GATED_BWD, ids=lambda v: str(v) if isinstance(v, int) else "")
def test_gated_linear_backward_paths(M, I, H, input_kernel, weight_kernel, dtype):
    log("gated backward path %dx%dx%d %s" % (M, I, H, dtype))
    x, w = make((M, H), dtype, 21), make((2 * I, H), dtype, 22, H ** -0.5)
    gu, dh = make((M, 2 * I), dtype, 23, 1.5), make((M, I), dtype, 24, 0.5)
    dx, dw = Guarded(M, H, TYPES[dtype]), Guarded(2 * I, H, TYPES[dtype])
    args = dev(dh, 1, 5), dev(x, 3), w.cuda(), dev(gu, 7, 1)
    got, names = launched(lambda: gr.gated_linear_backward(*args, act="silu", bias=True, dx_out=dx.view, dw_out=dw.view))
    refs, bounds = train_ref.gated_backward(dh, x, w, gu, "silu")
    for g, r, b in zip((dx.check(), dw.check(), got[2].cpu()), refs, bounds):
        check16(g, r, TYPES[dtype], b)
    check_launched(names, *[k(dtype) for k in (input_kernel, weight_kernel) if k])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,kernel", [(333, 1001, 2080, lambda e: stream(e, 4, 64)), (65, 130, 96, lambda e: stream(e, 8, 64)),
                                          (1500, 1501, 1500, lambda e: tile128(e, True))], ids=lambda v: str(v) if isinstance(v, int) else "")
def test_linear_backward_in_one_launch(M, N, K, kernel, dtype):
    """Both products and the bias's sums."""
    log("linear backward in one launch %dx%dx%d %s" % (M, N, K, dtype))
    dy, x, w = make((M, N), dtype, 14), make((M, K), dtype, 15), make((N, K), dtype, 16, K ** -0.5)
    dys, xs, ws = dy.cuda(), x.cuda(), w.cuda()
    got, names = launched(lambda: gr.linear_backward(dys, xs, ws, bias=True))
    refs, bounds = train_ref.linear_backward(dy, x, w)
    for g, r, b in zip(got, refs, bounds):
        check16(g.cpu(), r, TYPES[dtype], b)
    check_launched(names, kernel(own("Two", dtype)))


# ---- sandwich norm -----------------------------------------------------------------------------

# rows, columns, threads for a row and chunks of 8 columns per thread, forward and backward
NORM = [(2100, 333, (64, 1), (64, 1)), (2100, 200, (64, 1), (64, 1)), (520, 600, (128, 1), (128, 1)), (520, 601, (128, 1), (128, 1)),
        (520, 1200, (256, 1), (256, 1)), (520, 1201, (256, 1), (256, 1)), (520, 2600, (256, 2), (512, 1)), (520, 2601, (256, 2), (512, 1)),
        (260, 8000, (512, 2), (1024, 1)), (260, 8001, (512, 2), (1024, 1)), (260, 12000, (1024, 2), (1024, 2)),
        (260, 12001, (1024, 2), (1024, 2)), (260, 20000, (1024, 4), (1024, 4)), (260, 32767, (1024, 4), (1024, 4))]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gates", ["none", "one for each row"])
@pytest.mark.parametrize("M,N,forward,backward", NORM, ids=lambda v: str(v) if isinstance(v, int) else "")
def test_sandwich_norm_paths(M, N, forward, backward, gates, dtype):
    """Each width with whole and with ragged chunks, with rows of one gate to a workgroup and with more gates than workgroups."""
    log("norm path %dx%d gates %s %s" % (M, N, gates, dtype))
    kind, split, whole = TYPES[dtype], gates == "none", "true" if N % 8 == 0 else "false"
    y, res, dt, dn = (make((M, N), dtype, 40 + i) for i in range(4))
    w, next_w = ((make((N,), torch.float64, 50 + i, 0.3) + 1).to(kind) for i in range(2))
    gate = None if split else make((M, N), dtype, 52)
    on = [None if t is None else t.cuda() for t in (y, res, w, next_w, gate, dt, dn)]
    total, normed = Guarded(M, N, kind), Guarded(M, N, kind)
    _, names = launched(lambda: gr.sandwich_norm(*on[:5], scale=0.5, eps=1e-5, total_out=total.view, normed_out=normed.view))
    ref, bound, rel = train_ref.sandwich(y, res, w, next_w, gate, 0.5, 1e-5)
    total, normed = total.check(), normed.check()
    check16(total, ref, kind, bound)
    ref = train_ref.next_norm(total, next_w, 1e-5)
    check16(normed, ref, kind, ref.abs() * rel)
    check_launched(names, "sandwich::forward_kernel<%s, %d, %d, %s>" % (ELEM[dtype], *forward, whole))
    t = total.cuda()
    got, names = launched(lambda: gr.sandwich_norm_backward(on[5], on[6], on[0], t, *on[2:5], scale=0.5, eps=1e-5))
    ref = train_ref.sandwich_backward(dt, dn, y, total, w, next_w, gate, 0.5, 1e-5)
    for g, rb in zip(got, ref.values()):
        assert (g is None) == (rb is None)
        if g is not None:
            check16(g.cpu(), rb[0], kind, rb[1])
    check_launched(names, "sandwich::backward_kernel<%s, %d, %d, %s, %s>" % (ELEM[dtype], *backward, "true" if split else "false", whole))


# ---- orthogonalised update -----------------------------------------------------------------------

# batch, rows, cols, the tiles and whether those of A and B, of X and of the result are ragged. The sides that the products
# see are padded to multiples of 64, the result's are not
ORTHO = [(14, 1024, 1024, tile256, False, False, False), (10, 1100, 2100, tile256, True, True, True),
         (10, 2100, 1100, tile256, True, True, True), (5, 640, 768, tile128, False, False, False),
         (5, 700, 900, tile128, True, True, True), (5, 900, 700, tile128, True, True, True)]


@pytest.mark.parametrize("batch,rows,cols,tile,symmetric,product,result", ORTHO, ids=lambda v: str(v) if type(v) is int else "")
def test_orthogonalize_paths(batch, rows, cols, tile, symmetric, product, result):
    """Two steps, so that the products of a step that is not the last run too. The bound is the one for the fp16 operands'
    roundings: what they move the fp64 form by, twice for other places of the same size, and half a bfloat16 step."""
    log("ortho path %d %dx%d" % (batch, rows, cols))
    g = torch.randn(batch, rows, cols, generator=torch.Generator().manual_seed(31))
    g[1, 5, 7] = float("nan")
    buf = torch.full((batch, rows + 1, cols + 3 + cols % 2), 77.0, dtype=torch.bfloat16, device="cuda")
    out, update = buf[:, :rows, 1:cols + 1], g.cuda()
    _, names = launched(lambda: gr.orthogonalize(update, steps=2, scale=0.5, out=out))
    for i in (0, batch // 2, batch - 1):
        ref = train_ref.newton_schulz(g[i], 2)
        held = train_ref.newton_schulz(g[i], 2, rounded=True)
        got = out[i].cpu().double() / 0.5
        assert (got - ref).norm() <= 2 * (held - ref).norm() + 2.0 ** -8 * ref.norm(), i
        # no part of the matrix is off by more than its share: rows and columns of 64
        for r in range(0, rows, 64):
            part = slice(r, r + 64)
            assert (got - ref)[part].norm() <= 4 * (held - ref)[part].norm() + 2.0 ** -8 * ref[part].norm(), (i, r)
        for c in range(0, cols, 64):
            part = (slice(None), slice(c, c + 64))
            assert (got - ref)[part].norm() <= 4 * (held - ref)[part].norm() + 2.0 ** -8 * ref[part].norm(), (i, c)
    assert bool(out[1].isnan().all()) and bool(out[2:].isfinite().all()) and bool(out[0].isfinite().all())
    out.fill_(77.0)
    assert bool((buf == 77).all())
    half, bf16 = ELEM["f16"], ELEM["bf16"]
    check_launched(names, tile("gr::own::Poly<%s, %s, true>" % (half, half), symmetric),
                   tile("gr::own::Poly<%s, %s, false>" % (half, half), product),
                   tile("gr::own::Poly<%s, %s, false>" % (half, bf16), result))
