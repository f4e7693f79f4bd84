"""GPU tests of the training operators against plain fp64 forms (train_ref): sizes where each path begins and ends, odd
sizes, row pitches and addresses, every activation, gradients one by one, batches, graphs and streams."""
import pytest
import torch

import dense_gemm_epilogue_tiled_amd as gr
import train_ref
from gpu_util import log
from mx_ref import check16
from train_ref import TYPES, make

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid", "tanh")


def dev(t, pad=0, offset=0):
    """t on the GPU; its rows `pad` elements further apart and its first `offset` elements behind a 256-byte border, in
    a buffer of NaN."""
    if t is None:
        return None
    if not pad and not offset:
        return t.cuda()
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + offset + 64,), float("nan"), dtype=t.dtype, device="cuda")
    v = torch.as_strided(buf, (rows, cols), (cols + pad, 1), offset)
    v.copy_(t)
    return v


def guarded(rows, cols, dtype, pad):
    """An output view and its buffer, filled with a sentinel."""
    buf = torch.full((rows + 2, cols + pad), 77.0, dtype=dtype, device="cuda")
    return buf[1:rows + 1, :cols], buf


def untouched(buf, rows, cols):
    b = buf.float().cpu()
    assert bool((b[0] == 77).all()) and bool((b[rows + 1:] == 77).all()) and bool((b[:, cols:] == 77).all())


# ---- gated linear ------------------------------------------------------------------------

# M, I, H: the kernel for up to 4 tokens, the small-M stream (H % 256 == 0), streamed blocks, 128 x 128 tiles with ragged
# edges, 256 x 256 tiles of one strip, packed H (test_parity_gpu_train_paths.py has sizes for each kernel by name)
GATED = [(1, 64, 256), (1, 33, 512), (16, 70, 256), (2, 5, 256), (3, 40, 288), (17, 33, 96), (64, 32, 32), (65, 100, 320),
         (130, 31, 64), (5, 1, 32), (200, 2100, 64), (129, 2049, 160), (257, 8200, 64), (512, 16384, 64), (300, 9000, 192),
         (1, 40, 7), (9, 70, 100), (70, 20, 33), (300, 8300, 90), (4, 8, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,I,H", GATED)
def test_gated_linear(M, I, H, dtype):
    log("gated %dx%dx%d %s" % (M, I, H, dtype))
    x, w = make((M, H), dtype, M + H), make((2 * I, H), dtype, I + 7, 1.5 / max(H, 1) ** 0.5)
    b = make((2 * I,), dtype, 5) if I % 2 else None
    h, gu = gr.gated_linear(x.cuda(), w.cuda(), None if b is None else b.cuda(), act="silu", keep=True)
    alone, none = gr.gated_linear(x.cuda(), w.cuda(), None if b is None else b.cuda(), act="silu")
    assert none is None and torch.equal(h, alone)
    ref, bound, ref_gu, bound_gu = train_ref.gated(x, w, b, "silu")
    check16(h.cpu(), ref, h.dtype, bound)
    check16(gu.cpu(), ref_gu, gu.dtype, bound_gu)


@pytest.mark.parametrize("M,I,H", [(3, 40, 256), (70, 64, 64), (300, 8200, 64)])
@pytest.mark.parametrize("name", ACTS)
def test_gated_linear_activations(name, M, I, H):
    x, w, b = make((M, H), "f16", 1), make((2 * I, H), "f16", 2, 3 / H ** 0.5), make((2 * I,), "f16", 3)
    h, _ = gr.gated_linear(x.cuda(), w.cuda(), b.cuda(), act=name)
    ref, bound, _, _ = train_ref.gated(x, w, b, name)
    check16(h.cpu(), ref, h.dtype, bound)


@pytest.mark.parametrize("M,I,H", [(2, 40, 256), (40, 50, 64), (140, 70, 96), (300, 8200, 64), (6, 40, 50)])
@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 0), (1, 5)])
def test_gated_linear_pitches(M, I, H, pad, offset):
    """Rows apart, at any address, with NaN between them; nothing is written beside the outputs."""
    log("gated pitches %dx%dx%d pad %d offset %d" % (M, I, H, pad, offset))
    x, w = make((M, H), "bf16", 11), make((2 * I, H), "bf16", 12, H ** -0.5)
    out, out_buf = guarded(M, I, torch.bfloat16, pad)
    gu, gu_buf = guarded(M, 2 * I, torch.bfloat16, pad)
    got = gr.gated_linear(dev(x, pad, offset), dev(w, pad, offset), act="gelu", keep=True, out=out, gu_out=gu)
    assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == gu.data_ptr()
    ref, bound, ref_gu, bound_gu = train_ref.gated(x, w, None, "gelu")
    check16(out.cpu(), ref, out.dtype, bound)
    check16(gu.cpu(), ref_gu, gu.dtype, bound_gu)
    untouched(out_buf, M, I)
    untouched(gu_buf, M, 2 * I)


def test_gated_linear_keeps_nan_and_infinity_in_their_places():
    M, I, H = 70, 64, 64
    x, w = make((M, H), "bf16", 21), make((2 * I, H), "bf16", 22, 0.1)
    x[5, 3], x[9, 1] = float("nan"), float("inf")
    h, gu = gr.gated_linear(x.cuda(), w.cuda(), act="relu", keep=True)
    bad = ~torch.isfinite(gu.cpu()).all(1)
    assert bad.nonzero().flatten().tolist() == [5, 9]
    assert bool(torch.isfinite(h.cpu()[[r for r in range(M) if r not in (5, 9)]]).all())


# ---- gradients of linear layers -----------------------------------------------------------

# M, N, K
LINEAR = [(1, 64, 64), (1, 1, 1), (3, 70, 33), (64, 64, 128), (65, 100, 96), (200, 1001, 72), (333, 130, 520), (100, 40, 2080),
          (1000, 96, 64), (2304, 2304, 64), (300, 2500, 2600), (2000, 64, 3), (4, 4096, 4100)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_backward(M, N, K, dtype):
    log("linear backward %dx%dx%d %s" % (M, N, K, dtype))
    dy, x, w = make((M, N), dtype, 31), make((M, K), dtype, 32), make((N, K), dtype, 33, K ** -0.5)
    got = gr.linear_backward(dy.cuda(), x.cuda(), w.cuda(), bias=True)
    refs, bounds = train_ref.linear_backward(dy, x, w)
    for g, r, b in zip(got, refs, bounds):
        check16(g.cpu(), r, g.dtype, b)


def test_linear_backward_one_by_one():
    """Each gradient alone is the one of the whole call; what is not asked for is None."""
    dy, x, w = make((77, 130), "bf16", 41).cuda(), make((77, 96), "bf16", 42).cuda(), make((130, 96), "bf16", 43).cuda()
    dx, dw, db = gr.linear_backward(dy, x, w, bias=True)
    only = gr.linear_backward(dy, None, w, weight_grad=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    only = gr.linear_backward(dy, x, w, input_grad=False)
    assert only[0] is None and torch.equal(only[1], dw) and only[2] is None
    only = gr.linear_backward(dy, None, w, bias=True, input_grad=False, weight_grad=False)
    assert only[0] is None and only[1] is None and torch.equal(only[2], db)
    assert gr.linear_backward(dy, None, w, input_grad=False, weight_grad=False) == (None, None, None)


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 0), (1, 5)])
@pytest.mark.parametrize("M,N,K", [(70, 96, 64), (300, 2304, 2304), (40, 33, 50)])
def test_linear_backward_pitches(M, N, K, pad, offset):
    log("linear backward pitches %dx%dx%d pad %d offset %d" % (M, N, K, pad, offset))
    dy, x, w = make((M, N), "bf16", 51), make((M, K), "bf16", 52), make((N, K), "bf16", 53, K ** -0.5)
    dx, dx_buf = guarded(M, K, torch.bfloat16, pad)
    dw, dw_buf = guarded(N, K, torch.bfloat16, pad)
    gr.linear_backward(dev(dy, pad, offset), dev(x, pad, offset), dev(w, pad, offset), dx_out=dx, dw_out=dw)
    refs, bounds = train_ref.linear_backward(dy, x, w)
    check16(dx.cpu(), refs[0], dx.dtype, bounds[0])
    check16(dw.cpu(), refs[1], dw.dtype, bounds[1])
    untouched(dx_buf, M, K)
    untouched(dw_buf, N, K)


def test_gradients_without_tokens_are_zero():
    w = make((64, 32), "bf16", 61).cuda()
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    dx, dw, db = gr.linear_backward(none, x, w, bias=True)
    assert dx.shape == (0, 32) and not dw.any() and not db.any()
    gu = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    dx, dw, db = gr.gated_linear_backward(none[:, :32], x, w, gu, bias=True)
    assert dx.shape == (0, 32) and dw.shape == (64, 32) and not dw.any() and not db.any()
    y = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(32, dtype=torch.bfloat16, device="cuda")
    got = gr.sandwich_norm_backward(y, y, y, y, one, one, one)
    assert got[0].shape == got[1].shape == (0, 32) and not any(bool(g.any()) for g in got[2:])


def test_gradients_of_empty_sides():
    dy = make((5, 64), "bf16", 62).cuda()
    dx, dw, db = gr.linear_backward(dy, torch.empty(5, 0, dtype=dy.dtype, device="cuda"),
                                    torch.empty(64, 0, dtype=dy.dtype, device="cuda"), bias=True)
    assert dx.shape == (5, 0) and dw.shape == (64, 0)
    check16(db.cpu(), dy.cpu().double().sum(0), db.dtype, dy.cpu().double().abs().sum(0) * train_ref.sum_bound(5))
    x = make((5, 32), "bf16", 63).cuda()
    dx, dw, db = gr.linear_backward(dy[:, :0], x, torch.empty(0, 32, dtype=dy.dtype, device="cuda"), bias=True)
    assert not dx.any() and dw.shape == (0, 32) and db.shape == (0,)


# ---- gradients of the gated linear layer ---------------------------------------------------

# M, I, H
GATED_BWD = [(1, 64, 256), (2, 33, 64), (17, 100, 50), (64, 32, 96), (130, 70, 128), (333, 1201, 72), (300, 1300, 2600), (2304, 1152, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,I,H", GATED_BWD)
def test_gated_linear_backward(M, I, H, dtype):
    log("gated backward %dx%dx%d %s" % (M, I, H, dtype))
    x, w = make((M, H), dtype, 71), make((2 * I, H), dtype, 72, H ** -0.5)
    gu, dh = make((M, 2 * I), dtype, 73, 1.5), make((M, I), dtype, 74, 0.5)
    got = gr.gated_linear_backward(dh.cuda(), x.cuda(), w.cuda(), gu.cuda(), act="silu", bias=True)
    refs, bounds = train_ref.gated_backward(dh, x, w, gu, "silu")
    for g, r, b in zip(got, refs, bounds):
        check16(g.cpu(), r, g.dtype, b)


@pytest.mark.parametrize("name", ACTS)
def test_gated_linear_backward_activations(name):
    """Every activation's derivative over its whole range, tails and zero among it; where dg or du leaves fp16's range
    the sums with it are infinite or NaN, and no others."""
    M, I, H = 64, 40, 64
    x, w = make((M, H), "f16", 81), make((2 * I, H), "f16", 82, H ** -0.5)
    gu, dh = make((M, 2 * I), "f16", 83), make((M, I), "f16", 84)
    gu[:, :I] = torch.linspace(-30, 30, M * I).reshape(M, I).half()
    gu[3, 5], gu[4, 6], gu[5, 7] = 0.0, 60000.0, -60000.0
    got = gr.gated_linear_backward(dh.cuda(), x.cuda(), w.cuda(), gu.cuda(), act=name, bias=True)
    refs, bounds = train_ref.gated_backward(dh, x, w, gu, name)
    for g, r, b in zip(got, refs, bounds):
        finite = r.isfinite()
        assert torch.equal(g.cpu().isfinite() | (r.abs() > 60000), finite | (r.abs() > 60000))
        check16(g.cpu()[finite], r[finite], g.dtype, b[finite])


def test_gated_backward_of_far_gates_is_finite():
    """Gates at the ends of bfloat16's range: derivatives are 0, 1 and nothing else."""
    for name in ACTS:
        gu = torch.tensor([[3e38, -3e38, 1e20, -1e20] + [1.0] * 4], dtype=torch.bfloat16)
        dh = torch.ones(1, 4, dtype=torch.bfloat16)
        w = torch.zeros(8, 32, dtype=torch.bfloat16)
        w[:4] = 1.0
        dx, _, db = gr.gated_linear_backward(dh.cuda(), None, w.cuda(), gu.cuda(), act=name, bias=True, weight_grad=False)
        want = {"none": [1, 1, 1, 1], "sigmoid": [0] * 4, "tanh": [0] * 4}.get(name, [1, 0, 1, 0])
        assert db[:4].float().tolist() == want, (name, db)
        assert dx.float().tolist() == [[float(sum(want))] * 32], name


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gated_backward_against_differences(name):
    """Forward and backward passes together: a gradient's product with a direction is the difference quotient of the fp64
    form at the kept values, and the forward pass's h is that form's."""
    M, I, H = 33, 48, 64
    x, w = make((M, H), "f16", 91), make((2 * I, H), "f16", 92, H ** -0.5)
    dh = make((M, I), "f16", 93)
    _, gu = gr.gated_linear(x.cuda(), w.cuda(), act=name, keep=True)
    dx, dw, _ = gr.gated_linear_backward(dh.cuda(), x.cuda(), w.cuda(), gu, act=name)

    def value(x, w):
        g, u = (x @ w.T).chunk(2, -1)
        return (train_ref.act(g, name) * u * dh.double()).sum()

    for leaf, grad in ((x, dx), (w, dw)):
        v = make(leaf.shape, torch.float64, 94)
        at, e = leaf.double(), 1e-4
        up = value(at + e * v, w.double()) if leaf is x else value(x.double(), at + e * v)
        down = value(at - e * v, w.double()) if leaf is x else value(x.double(), at - e * v)
        # what is rounded to 11 bits in between: gu, dg and du, the gradient: 4 half steps of each product's magnitude, of
        # which the direction's signs leave the root over all the elements
        got = (grad.cpu().double() * v).sum()
        size = (grad.cpu().double() * v).norm()
        assert abs(got - (up - down) / (2 * e)) <= 6 * 4 * 2.0 ** -11 * size, (name, got, (up - down) / (2 * e))


# ---- sandwich norm ---------------------------------------------------------------------------

NORM = [(1, 1), (1, 4096), (3, 7), (5, 64), (8, 513), (7, 1024), (600, 520), (9, 1025), (4, 2049), (300, 4000), (6, 4097), (260, 8192),
        (3, 8200), (2, 16384), (2, 16400), (1, 32768), (1100, 8)]


def norm_inputs(M, N, dtype, G, seed):
    w, next_w = make((N,), dtype, seed, 0.3) + 1, make((N,), dtype, seed + 1, 0.3) + 1
    gate = None if G is None else make((N,) if G == 0 else (G, N), dtype, seed + 2)
    return make((M, N), dtype, seed + 3), make((M, N), dtype, seed + 4, 2.0), w.to(TYPES[dtype]), next_w.to(TYPES[dtype]), gate


def some_gate(M):
    """None, N values, a row for every row, or one for every half or third."""
    return [None, 0, M, 2 if M % 2 == 0 else 3 if M % 3 == 0 else 1][M % 4]


def check_sandwich(got, y, res, w, next_w, gate, scale, eps):
    total, normed = got
    ref, bound, rel = train_ref.sandwich(y, res, w, next_w, gate, scale, eps)
    check16(total.cpu(), ref, total.dtype, bound)
    if normed is not None:
        n = train_ref.next_norm(total.cpu(), next_w, eps)
        check16(normed.cpu(), n, normed.dtype, n.abs() * rel)


def gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", NORM)
def test_sandwich_norm(M, N, dtype):
    log("sandwich %dx%d %s" % (M, N, dtype))
    y, res, w, next_w, gate = norm_inputs(M, N, dtype, some_gate(M), 100)
    got = gr.sandwich_norm(*gpu(y, res, w, next_w, gate), scale=0.5, eps=1e-5)
    check_sandwich(got, y, res, w, next_w, gate, 0.5, 1e-5)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", NORM)
def test_sandwich_norm_backward(M, N, dtype):
    log("sandwich backward %dx%d %s" % (M, N, dtype))
    y, total, w, next_w, gate = norm_inputs(M, N, dtype, some_gate(M), 110)
    dt, dn = make((M, N), dtype, 120), make((M, N), dtype, 121)
    got = gr.sandwich_norm_backward(*gpu(dt, dn, y, total, w, next_w, gate), scale=0.5, eps=1e-5)
    ref = train_ref.sandwich_backward(dt, dn, y, total, w, next_w, gate, 0.5, 1e-5)
    for g, (name, rb) in zip(got, ref.items()):
        assert (g is None) == (rb is None), name
        if g is not None:
            check16(g.cpu().reshape(rb[0].shape), rb[0], g.dtype, rb[1])
            assert g.shape == {"dw": w, "dnext_w": next_w, "dgate": gate}.get(name, y).shape, name


@pytest.mark.parametrize("G", [1, 6, 1200, 2400])
def test_sandwich_norm_gates(G):
    """From one gate for all rows to one each: more gates than workgroups among them."""
    M, N = 2400, 72
    y, res, w, next_w, gate = norm_inputs(M, N, "bf16", G, 130)
    check_sandwich(gr.sandwich_norm(*gpu(y, res, w, next_w, gate)), y, res, w, next_w, gate, 1.0, 1e-6)
    dt, dn = make((M, N), "bf16", 140), make((M, N), "bf16", 141)
    got = gr.sandwich_norm_backward(*gpu(dt, dn, y, res, w, next_w, gate))
    ref = train_ref.sandwich_backward(dt, dn, y, res, w, next_w, gate, 1.0, 1e-6)
    for g, rb in zip(got, ref.values()):
        check16(g.cpu(), rb[0], g.dtype, rb[1])


@pytest.mark.parametrize("what", ["no weights", "no next norm", "no gate", "dtotal only", "dnormed only", "nothing learned"])
def test_sandwich_norm_parts(what):
    M, N = 20, 600
    y, res, w, next_w, gate = norm_inputs(M, N, "f16", 4, 150)
    dt, dn = make((M, N), "f16", 160), make((M, N), "f16", 161)
    norm = True
    if what in ("no weights", "nothing learned"):
        w = next_w = None
    if what in ("no gate", "nothing learned"):
        gate = None
    if what == "no next norm":
        norm, next_w = False, None
    if what in ("dtotal only", "no next norm"):
        dn = None
    if what == "dnormed only":
        dt = None
    got = gr.sandwich_norm(*gpu(y, res, w, next_w, gate), scale=-2.0, next_norm=norm)
    assert (got[1] is not None) == norm
    check_sandwich(got, y, res, w, next_w, gate, -2.0, 1e-6)
    got = gr.sandwich_norm_backward(*gpu(dt, dn, y, res, w, next_w, gate), scale=0.25)
    ref = train_ref.sandwich_backward(dt, dn, y, res, w, next_w, gate, 0.25, 1e-6)
    for g, rb in zip(got, ref.values()):
        assert (g is None) == (rb is None)
        if g is not None:
            check16(g.cpu(), rb[0], g.dtype, rb[1])


@pytest.mark.parametrize("N", [70, 1000, 2100, 9000])
def test_sandwich_norm_in_place_and_apart(N):
    """Outputs on the inputs, and inputs with rows apart: the same bits."""
    y, res, w, next_w, gate = gpu(*norm_inputs(12, N, "bf16", 3, 170))
    total, normed = gr.sandwich_norm(y, res, w, next_w, gate)
    for first, second in (("r", "y"), ("y", "r"), ("r", None), (None, "r"), (None, "y")):
        y2, r2 = y.clone(), res.clone()
        on = {"y": y2, "r": r2, None: None}
        a, b = gr.sandwich_norm(y2, r2, w, next_w, gate, total_out=on[first], normed_out=on[second])
        assert torch.equal(a, total) and torch.equal(b, normed), (first, second)
    out, buf = guarded(12, N, torch.bfloat16, 5)
    a, b = gr.sandwich_norm(dev(y, 3, 1), dev(res, 1, 7), w, next_w, gate, total_out=out)
    assert torch.equal(a, total) and torch.equal(b, normed)
    untouched(buf, 12, N)
    dt, dn = make((12, N), "bf16", 180).cuda(), make((12, N), "bf16", 181).cuda()
    whole = gr.sandwich_norm_backward(dt, dn, y, total, w, next_w, gate)
    apart = gr.sandwich_norm_backward(dev(dt, 3, 1), dev(dn, 5, 3), dev(y, 1, 1), dev(total, 9, 2), w, next_w, dev(gate, 2, 1))
    for a, b in zip(whole, apart):
        assert torch.equal(a, b)


def test_sandwich_norm_of_zeros():
    """Rows of zeros: eps alone is under the root."""
    y = torch.zeros(4, 96, dtype=torch.bfloat16, device="cuda")
    total, normed = gr.sandwich_norm(y, y, eps=1e-6)
    assert not total.any() and not normed.any()
    d = make((4, 96), "bf16", 190)
    dy, dres, _, _, _ = gr.sandwich_norm_backward(d.cuda(), d.cuda(), y, y, eps=1e-6)
    ref = train_ref.sandwich_backward(d, d, y.cpu(), y.cpu(), None, None, None, 1.0, 1e-6)
    check16(dres.cpu(), *[ref["dresidual"][0], dres.dtype, ref["dresidual"][1]])
    check16(dy.cpu(), *[ref["dy"][0], dy.dtype, ref["dy"][1]])


# ---- orthogonalised update ---------------------------------------------------------------------

def check_ortho(got, update, steps=5, coefficients=train_ref.QUINTIC, scale=1.0):
    """The fp16 operands' roundings move the result by as much as they move it in fp64, to within a factor of two in the
    2-norm (roundings of the same sizes at other places); half a bfloat16 step is added."""
    ref = train_ref.newton_schulz(update, steps, coefficients)
    held = train_ref.newton_schulz(update, steps, coefficients, rounded=True)
    err = (got.double().cpu() - scale * ref).norm()
    allowed = scale * (2 * (held - ref).norm() + 2.0 ** -8 * ref.norm())
    log("ortho %s: %.2e of %.2e" % (tuple(update.shape), err / (scale * ref.norm()), allowed / (scale * ref.norm())))
    assert got.dtype == torch.bfloat16 and got.shape == update.shape
    assert err <= allowed, (float(err), float(allowed))


ORTHO = [(1, 1), (1, 300), (300, 1), (16, 16), (64, 64), (63, 65), (100, 37), (130, 700), (640, 200), (1100, 1300), (1300, 1100), (2200, 2176)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", ORTHO)
def test_orthogonalize(rows, cols, dtype):
    log("ortho %dx%d %s" % (rows, cols, dtype))
    g = make((rows, cols), dtype, rows + cols, 1e-2)
    check_ortho(gr.orthogonalize(g.cuda()), g)


@pytest.mark.parametrize("batch,rows,cols", [(3, 64, 130), (5, 200, 70), (2, 600, 1000), (9, 256, 256), (2, 1100, 1100)])
def test_orthogonalize_batch(batch, rows, cols):
    """A batch is its matrices one by one, to the order of the sums."""
    log("ortho batch %d %dx%d" % (batch, rows, cols))
    g = make((batch, rows, cols), torch.float32, 7) * torch.logspace(-8, 8, batch)[:, None, None]
    got = gr.orthogonalize(g.cuda())
    for i in range(batch):
        check_ortho(got[i], g[i])


def test_orthogonalize_places():
    """Rows and matrices apart, at any address, next to NaN; nothing is written beside the output."""
    g = make((3, 70, 90), torch.bfloat16, 8)
    want = gr.orthogonalize(g.cuda())
    buf = torch.full((3 * 75 * 97 + 1,), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.as_strided(buf, (3, 70, 90), (75 * 97, 97, 1), 1)
    v.copy_(g)
    out = torch.full((3, 72, 95), 77.0, dtype=torch.bfloat16, device="cuda")
    gr.orthogonalize(v, out=out[:, 1:71, 2:92])
    assert torch.equal(out[:, 1:71, 2:92], want)
    out[:, 1:71, 2:92] = 77.0
    assert bool((out == 77).all())


def test_orthogonalize_arguments():
    g = make((96, 160), torch.float32, 9)
    check_ortho(gr.orthogonalize(g.cuda(), steps=1), g, steps=1)
    check_ortho(gr.orthogonalize(g.cuda(), steps=8, coefficients=(15 / 8, -10 / 8, 3 / 8), scale=0.25), g, 8,
                (15 / 8, -10 / 8, 3 / 8), 0.25)
    # singular values: all between the polynomial's ends near 1
    s = torch.linalg.svdvals(gr.orthogonalize(g.cuda()).cpu().double())
    assert 0.65 < float(s.min()) and float(s.max()) < 1.25


def test_orthogonalize_special_values():
    zero = torch.zeros(70, 70, device="cuda")
    assert not gr.orthogonalize(zero).any()
    for bad in (float("nan"), float("inf")):
        g = make((2, 70, 40), torch.float32, 10)
        g[0, 3, 4] = bad
        got = gr.orthogonalize(g.cuda())
        assert bool(got[0].isnan().all()) and bool(got[1].isfinite().all())
    for scale in (1e-25, 1e18, 1e30):  # far from where fp32 squares have their place
        g = make((40, 70), torch.float32, 11) * scale
        if scale < 1:
            got = gr.orthogonalize(g.cuda(), eps=0.0)
        else:
            got = gr.orthogonalize(g.cuda())
        ref = train_ref.newton_schulz(g, 5, eps=0.0)
        assert (got.cpu().double() - ref).norm() <= 0.01 * ref.norm()


# ---- all together: graphs, streams ---------------------------------------------------------------

def training_step(x, res, w13, w2, w, next_w, gate, dtotal, dnormed):
    """A block's forward and backward pass and its weights' updates, as a training loop calls them."""
    h, gu = gr.gated_linear(x, w13, act="silu", keep=True)
    y = gr.linear(h, w2)
    total, normed = gr.sandwich_norm(y, res, w, next_w, gate, scale=0.5)
    dy, dres, dw, dnext, dgate = gr.sandwich_norm_backward(dtotal, dnormed, y, total, w, next_w, gate, scale=0.5)
    dh, dw2, _ = gr.linear_backward(dy, h, w2)
    dx, dw13, _ = gr.gated_linear_backward(dh, x, w13, gu, act="silu")
    return [h, gu, y, total, normed, dy, dres, dw, dnext, dgate, dh, dw2, dx, dw13, gr.orthogonalize(dw13),
            gr.orthogonalize(dw2)]


def step_inputs(M, H, I, seed):
    return gpu(make((M, H), "bf16", seed), make((M, H), "bf16", seed + 1), make((2 * I, H), "bf16", seed + 2, H ** -0.5),
               make((H, I), "bf16", seed + 3, I ** -0.5), make((H,), "bf16", seed + 4), make((H,), "bf16", seed + 5),
               make((2, H), "bf16", seed + 6), make((M, H), "bf16", seed + 7, 0.1), make((M, H), "bf16", seed + 8, 0.1))


@pytest.mark.parametrize("M,H,I", [(2, 256, 128), (78, 200, 131), (600, 512, 1100)])
def test_training_step_in_a_graph(M, H, I):
    """Captured once, replayed on changing inputs between eager work: every replay gives the eager call's bits."""
    static = step_inputs(M, H, I, 300)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        training_step(*static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = training_step(*static)
    for k in range(3):
        fresh = step_inputs(M, H, I, 400 + 20 * k)
        want = training_step(*fresh)
        for s, f in zip(static, fresh):
            s.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Two steps at a time on streams of their own, workspaces and outputs apart."""
    inputs = [step_inputs(130, 256, 300, 500), step_inputs(64, 512, 130, 600)]
    want = [[t.clone() for t in training_step(*i)] for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, i in zip(streams, inputs):
            with torch.cuda.stream(s):
                got.append(training_step(*i))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_a_stream_given():
    x, w = make((70, 64), "bf16", 700).cuda(), make((80, 64), "bf16", 701).cuda()
    want, _ = gr.gated_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = gr.gated_linear(x, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_repeated_calls_give_the_same_bits():
    i = step_inputs(334, 520, 700, 800)
    first = [t.clone() for t in training_step(*i)]
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(training_step(*i), first))


# ---- the block that is trained --------------------------------------------------------------------

def test_trained_block_gradients():
    """feed_forward's forward and backward passes against the fp64 form of the whole block: what is rounded in between
    moves a gradient by a few roundings of 8 bits, in the 2-norm."""
    from dense_gemm_epilogue_tiled_amd import feed_forward as ff
    M, H, I = 96, 128, 200
    x, res = make((M, H), "bf16", 900), make((M, H), "bf16", 901, 2.0)
    weights = {"w13": make((2 * I, H), "bf16", 902, H ** -0.5), "w2": make((H, I), "bf16", 903, I ** -0.5),
               "norm": (make((H,), torch.float64, 904, 0.2) + 1).bfloat16(), "next_norm": (make((H,), torch.float64, 905, 0.2) + 1).bfloat16(),
               "gate": make((3, H), "bf16", 906)}
    dt, dn = make((M, H), "bf16", 907), make((M, H), "bf16", 908)
    on = {n: w.cuda() for n, w in weights.items()}
    (total, normed), kept = ff.train_forward(x.cuda(), res.cuda(), **on, scale=0.5)
    dx, dres, grads = ff.train_backward(dt.cuda(), dn.cuda(), kept, **on, scale=0.5)
    leaves = {"x": x, "res": res, **weights}
    leaves = {n: t.double().requires_grad_() for n, t in leaves.items()}
    g, u = (leaves["x"] @ leaves["w13"].T).chunk(2, -1)
    y = (train_ref.act(g, "silu") * u) @ leaves["w2"].T
    ref_total, _, _ = train_ref.sandwich(y, leaves["res"], leaves["norm"], None, leaves["gate"], 0.5, 1e-6)
    ref_normed = train_ref.next_norm(ref_total, leaves["next_norm"], 1e-6)
    ref = torch.autograd.grad((ref_total * dt.double()).sum() + (ref_normed * dn.double()).sum(), list(leaves.values()))
    got = [dx, dres, *grads.values()]
    step = 2.0 ** -8
    for name, a, b in [("total", total, ref_total), ("normed", normed, ref_normed), *zip(leaves, got, ref)]:
        # gu, h, y, total, dy, dh, dgu and the result: 8 roundings of half a step at most each, as if all fell together
        assert (a.double().cpu() - b.detach()).norm() <= 8 * step * b.detach().norm(), name


def test_training_demo_runs():
    from dense_gemm_epilogue_tiled_amd import feed_forward as ff
    weights, grads = ff._train_demo(40, 96, 130, 3)
    assert all(bool(t.isfinite().all()) for t in [*weights.values(), *grads.values()])


def test_update_matrix_moves_along_the_orthogonalised_momentum():
    from dense_gemm_epilogue_tiled_amd import feed_forward as ff
    w, grad, m = make((130, 70), "bf16", 950).cuda(), make((130, 70), "bf16", 951).cuda(), make((130, 70), torch.float32, 952).cuda()
    before, mom = w.clone(), m * 0.9 + grad
    ff.update_matrix(w, grad, m, 0.5, 0.9)
    assert torch.equal(m, mom)
    want = before.add(gr.orthogonalize(mom * 0.9 + grad, scale=(130 / 70) ** 0.5), alpha=-0.5)
    assert torch.equal(w, want)


# ---- corners ---------------------------------------------------------------------------------------

def test_gated_gradients_of_empty_sides():
    dh, x = torch.empty(5, 0, dtype=torch.bfloat16, device="cuda"), make((5, 32), "bf16", 970).cuda()
    w = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    dx, dw, db = gr.gated_linear_backward(dh, x, w, dh, bias=True)
    assert dx.shape == (5, 32) and not dx.any() and dw.shape == (0, 32) and db.shape == (0,)
    h, gu = gr.gated_linear(x, w, keep=True)
    assert h.shape == (5, 0) and gu.shape == (5, 0)
    dh, gu = make((70, 8), "bf16", 971), make((70, 16), "bf16", 972)
    no_x, no_w = torch.empty(70, 0, dtype=torch.bfloat16, device="cuda"), torch.empty(16, 0, dtype=torch.bfloat16, device="cuda")
    dx, dw, db = gr.gated_linear_backward(dh.cuda(), no_x, no_w, gu.cuda(), bias=True)
    assert dx.shape == (70, 0) and dw.shape == (16, 0)
    refs, bounds = train_ref.gated_backward(dh, torch.zeros(70, 1), torch.zeros(16, 1), gu, "silu")
    check16(db.cpu(), refs[2], db.dtype, bounds[2])


def far(t, pitch):
    """t's rows `pitch` elements apart, past 2^32 bytes in all."""
    buf = torch.empty(t.shape[0] * pitch, dtype=t.dtype, device="cuda")
    v = torch.as_strided(buf, t.shape, (pitch, 1))
    v.copy_(t)
    return v


def test_far_rows():
    """Rows 4 MB apart: offsets beyond 32 bits in every operand and output, on each kernel's tiles."""
    pitch = 1 << 21
    M, H, I = 1100, 64, 72
    x, w, dh = make((M, H), "bf16", 980).cuda(), make((2 * I, H), "bf16", 981, H ** -0.5).cuda(), make((M, I), "bf16", 982).cuda()
    want, want_gu = gr.gated_linear(x, w, keep=True)
    out = far(torch.zeros_like(want), pitch)
    got, gu = gr.gated_linear(far(x, pitch), w, keep=True, out=out, gu_out=far(torch.zeros_like(want_gu), pitch))
    assert torch.equal(got, want) and torch.equal(gu, want_gu)
    dx, dw, _ = gr.gated_linear_backward(dh, x, w, want_gu)
    a, b, _ = gr.gated_linear_backward(far(dh, pitch), far(x, pitch), w, gu, dx_out=out.as_strided((M, H), (pitch, 1)))
    assert torch.equal(a, dx) and torch.equal(b, dw)
    del out, got, gu
    y, res = make((M, I), "bf16", 983).cuda(), make((M, I), "bf16", 984).cuda()
    total, normed = gr.sandwich_norm(y, res)
    a, b = gr.sandwich_norm(far(y, pitch), far(res, pitch), total_out=far(torch.zeros_like(y), pitch))
    assert torch.equal(a, total) and torch.equal(b, normed)


def test_rows_beyond_one_launch():
    """More rows than one launch's threads: the last ones are computed too."""
    M, N = (1 << 22) + 5, 8
    y, res = torch.randn(M, N, device="cuda").bfloat16(), torch.randn(M, N, device="cuda").bfloat16()
    gate = torch.randn(3, N, device="cuda").bfloat16()
    assert M % 3 == 0
    total, normed = gr.sandwich_norm(y, res, gate=gate)
    tail = slice(M - 9, M)
    a, b = gr.sandwich_norm(y[tail], res[tail], gate=gate[2])
    assert torch.equal(total[tail], a) and torch.equal(normed[tail], b)


def test_wide_gates_of_few_tokens():
    """More columns than one pass of the kernel for few tokens takes."""
    M, I, H = 2, (1 << 23) + 77, 8
    x, w = make((M, H), "bf16", 990).cuda(), torch.randn(2 * I, H, device="cuda").bfloat16()
    h, _ = gr.gated_linear(x, w)
    at = torch.tensor([0, 1, 4095, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, I - 1], device="cuda")
    some, _ = gr.gated_linear(x, torch.cat((w[at], w[I + at])))
    assert torch.equal(h[:, at], some)


@pytest.mark.parametrize("M,N,K", [(6061, 320, 222), (8192, 70, 65), (5000, 128, 131), (20000, 64, 64)])
def test_linear_backward_of_many_tokens(M, N, K):
    """Few blocks and many tokens: the tokens are cut into ranges, whose sums a second pass adds."""
    log("many tokens %dx%dx%d" % (M, N, K))
    dy, x, w = make((M, N), "bf16", 1001), make((M, K), "bf16", 1002), make((N, K), "bf16", 1003, K ** -0.5)
    dw, dw_buf = guarded(N, K, torch.bfloat16, 3)
    got = gr.linear_backward(dy.cuda(), x.cuda(), w.cuda(), bias=True, dw_out=dw)
    refs, bounds = train_ref.linear_backward(dy, x, w)
    for g, r, b in zip(got, refs, bounds):
        check16(g.cpu(), r, g.dtype, b)
    untouched(dw_buf, N, K)
    assert torch.equal(gr.linear_backward(dy.cuda(), x.cuda(), w.cuda(), input_grad=False)[1], dw)


@pytest.mark.parametrize("batch,rows,cols", [(1, 33, 4001), (3, 3000, 64), (2, 100, 1500), (2, 1501, 120), (3, 191, 257), (1, 2000, 193),
                                             (40, 250, 300)])
def test_orthogonalize_of_a_narrow_side_up_to_256(batch, rows, cols):
    """Each of the kernel's widths, either way round, one and several blocks of columns to a workgroup; with the outputs
    apart at odd addresses, and a matrix of NaN beside the others."""
    log("ortho narrow %d %dx%d" % (batch, rows, cols))
    g = make((batch, rows, cols), torch.float32, 21)
    buf = torch.full((batch, rows + 1, cols + 3), 77.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :rows, 1:cols + 1]
    gr.orthogonalize(g.cuda(), out=out)
    for i in range(min(batch, 3)):
        check_ortho(out[i], g[i])
    want = out.clone()
    out.fill_(77.0)
    assert bool((buf == 77).all())
    g[0, 1, 2] = float("nan")
    got = gr.orthogonalize(g.cuda())
    assert bool(got[0].isnan().all()) and torch.equal(got[1:], want[1:])


@pytest.mark.parametrize("rows,cols", [(200, 1300), (1300, 200)])
def test_orthogonalize_of_a_narrow_side_arguments(rows, cols):
    """One step, which is the last; other coefficients, steps and a scale."""
    log("ortho narrow arguments %dx%d" % (rows, cols))
    g = make((rows, cols), torch.float32, 22)
    check_ortho(gr.orthogonalize(g.cuda(), steps=1), g, steps=1)
    check_ortho(gr.orthogonalize(g.cuda(), steps=8, coefficients=(15 / 8, -10 / 8, 3 / 8), scale=0.25), g, 8,
                (15 / 8, -10 / 8, 3 / 8), 0.25)


def test_small_gradients_and_narrow_updates_in_a_graph():
    """Ranges of tokens, two products in a launch, updates in two launches a step: replayed on new inputs, with eager
    calls in between, and the same bits as eager calls."""
    log("graph of small gradients and narrow updates")
    M, N, K = 5000, 200, 131
    dy, x = make((M, N), "bf16", 31).cuda(), make((M, K), "bf16", 32).cuda()
    w, a = make((N, K), "bf16", 33).cuda(), make((2, 160, 500), torch.float32, 34).cuda()

    def work():
        return (*gr.linear_backward(dy, x, w, bias=True), gr.orthogonalize(a))

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for seed in range(4):
        for t in (dy, x, w, a):
            t.copy_(make(tuple(t.shape), t.dtype, 40 + seed))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(held, work()):
            assert torch.equal(got, want)
