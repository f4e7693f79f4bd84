"""GPU tests of the training operators where a call has nothing to sum or leaves a type's range."""
import pytest
import torch

import dense_gemm_epilogue_tiled_amd as gr
import train_ref
from gpu_util import log
from mx_ref import check16
from train_ref import TYPES, make

pytestmark = pytest.mark.gpu

INF = float("inf")


def nans(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def norm_bwd_without_rows(N, w, gate, G, dw, dnext, dgate, fmt=gr.GR_FMT_BF16, ws=None):
    at = [None if t is None else t.data_ptr() for t in (w, w, gate if G else None, dw, dnext, dgate if G else None, ws)]
    return gr.sandwich_norm_bwd(0, N, None, N, None, N, None, N, None, N, *at[:3], G, N, 1.0, 1e-6, None, N, None, N, *at[3:6], N,
                                fmt, at[6], 0 if ws is None else ws.numel(), torch.cuda.current_stream().cuda_stream)


def used_memory():
    """Leaves the allocator's small free blocks full of NaN: an output that nothing writes shows."""
    blocks = [nans(n) for n in (64, 256, 2048, 20000) for _ in range(24)]
    torch.cuda.synchronize()
    del blocks


# ---- no rows -----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("G", [0, 1, 3])
@pytest.mark.parametrize("N", [1, 40, 1030])
def test_norm_gradients_without_rows_are_written(N, G, workspace, dtype):
    """Zeros, with a workspace and without: no rows need none."""
    log("norm without rows N %d G %d %s" % (N, G, dtype))
    kind = TYPES[dtype]
    w, gate = torch.ones(N, dtype=kind, device="cuda"), torch.ones(max(G, 1), N, dtype=kind, device="cuda")
    dw, dnext, dgate = nans(N, dtype=kind), nans(N, dtype=kind), nans(max(G, 1), N, dtype=kind)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda") if workspace else None
    assert gr.sandwich_norm_bwd_workspace_size(0, N, G) == (gr.GR_OK, 0)
    st = norm_bwd_without_rows(N, w, gate, G, dw, dnext, dgate, gr.GR_FMT_BF16 if dtype == "bf16" else gr.GR_FMT_F16, ws)
    assert st == gr.GR_OK
    for g in (dw, dnext, dgate)[:3 if G else 2]:
        assert bool((g == 0).all())


@pytest.mark.parametrize("G", [0, 1, 3])
def test_norm_gradients_without_rows_one_by_one(G):
    """Each sum alone; the others' places stay as they are."""
    N = 40
    w, gate = torch.ones(N, dtype=torch.bfloat16, device="cuda"), torch.ones(max(G, 1), N, dtype=torch.bfloat16, device="cuda")
    for wanted in range(3 if G else 2):
        out = [nans(N), nans(N), nans(max(G, 1), N)]
        given = [t if i == wanted else None for i, t in enumerate(out)]
        st = norm_bwd_without_rows(N, w, gate, G, *given)
        assert st == gr.GR_OK
        for i, t in enumerate(out):
            assert bool((t == 0).all() if i == wanted else t.isnan().all())


def test_helpers_gradients_without_rows_are_written():
    """Every gradient of a batch without tokens, in memory that held NaN."""
    w, y = torch.ones(64, 32, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    one, gates = torch.ones(32, dtype=torch.bfloat16, device="cuda"), torch.ones(5, 32, dtype=torch.bfloat16, device="cuda")
    gu = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    for gate in (None, one, gates):
        used_memory()
        got = gr.sandwich_norm_backward(y, y, y, y, one, one, gate)[2:]
        assert all(g is None if gate is None and i == 2 else bool((g == 0).all()) for i, g in enumerate(got))
    for call in (lambda out: gr.linear_backward(gu, y, w, bias=True, dw_out=out),
                 lambda out: gr.gated_linear_backward(y, y, w, gu, bias=True, dw_out=out)):
        used_memory()
        out = nans(64, 32)
        _, dw, db = call(out)
        assert dw.data_ptr() == out.data_ptr() and bool((dw == 0).all()) and bool((db == 0).all())


# ---- gates beyond the type's range ----------------------------------------------------------

# value and slope at -infinity and at +infinity
LIMITS = {"none": (-INF, 1, INF, 1), "relu": (0, 0, INF, 1), "gelu": (0, 0, INF, 1), "gelu_tanh": (0, 0, INF, 1), "silu": (0, 0, INF, 1),
          "sigmoid": (0, 0, 1, 0), "tanh": (-1, 0, 1, 0)}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", LIMITS)
def test_gated_backward_of_infinite_gates(name, dtype):
    """The activation's limits, and NaN for NaN alone."""
    low, low_slope, high, high_slope = LIMITS[name]
    gu = torch.tensor([[-INF, INF, float("nan"), 0.5] + [2.0] * 4], dtype=TYPES[dtype])
    dh, w = torch.full((1, 4), 0.5, dtype=TYPES[dtype]), torch.zeros(8, 32, dtype=TYPES[dtype])
    db = gr.gated_linear_backward(dh.cuda(), None, w.cuda(), gu.cuda(), act=name, bias=True, input_grad=False, weight_grad=False)[2].tolist()
    assert db[:2] == [low_slope * 1.0, high_slope * 1.0] and db[4:6] == [low * 0.5, high * 0.5], db
    assert db[2] != db[2] or name in ("relu", "none")  # the slopes of these are constants
    assert db[6] != db[6] or name == "relu" and db[6] == 0
    assert all(v == v for v in (db[3], db[7]))


@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu", "sigmoid"])
def test_gradients_of_gates_far_below_float16(name):
    """Gates whose sums are finite and beyond float16's range: the forward pass gives zeros there, and the gradients are
    finite and those of the sums."""
    M, I, H = 70, 40, 64
    log("far gates %s" % name)
    x, w, dh = make((M, H), "f16", 11), make((2 * I, H), "f16", 12, H ** -0.5), make((M, I), "f16", 13)
    x[:, 0], w[3, 0], w[7, 0] = 60.0, -2000.0, -30000.0
    h, gu = gr.gated_linear(x.cuda(), w.cuda(), act=name, keep=True)
    sums = x.double() @ w.double().T
    assert bool((gu[:, [3, 7]] == -INF).all()) and float(sums[:, [3, 7]].max()) < -65536
    assert bool(gu[:, [c for c in range(2 * I) if c not in (3, 7)]].isfinite().all()) and not h[:, [3, 7]].any()
    got = gr.gated_linear_backward(dh.cuda(), x.cuda(), w.cuda(), gu, act=name, bias=True)
    # at -100 as at the sums every value and slope is below 1e-40
    kept = gu.cpu().double()
    kept[:, [3, 7]] = -100.0
    refs, bounds = train_ref.gated_backward(dh, x, w, kept, name)
    for g, r, b in zip(got, refs, bounds):
        assert bool(r.isfinite().all())
        check16(g.cpu(), r, g.dtype, b)
    none = [3, 7, I + 3, I + 7]
    assert not got[1][none].any() and not got[2][none].any()


# ---- updates at the ends of the range without an eps ----------------------------------------

# one workgroup's, two launches a step, three launches a step; wide and tall
UPDATES = [(8, 8), (70, 70), (128, 500), (500, 100), (200, 1300), (1300, 150), (600, 700), (700, 600)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", UPDATES)
def test_zero_update_without_eps(rows, cols, dtype):
    """Zeros beside a matrix that is not: zeros, and the other's own result."""
    g = torch.stack((torch.zeros(rows, cols), make((rows, cols), torch.float32, 21))).to(dtype)
    got = gr.orthogonalize(g.cuda(), eps=0.0)
    assert bool((got[0] == 0).all())
    assert torch.equal(got[1], gr.orthogonalize(torch.stack((g[1], g[1])).cuda(), eps=0.0)[1])
    assert bool((gr.orthogonalize(g[:1].cuda(), eps=0.0) == 0).all())


@pytest.mark.parametrize("scale", [1e-44, 1e-41, 1e-37, 1e-36, 1e38])
@pytest.mark.parametrize("rows,cols", UPDATES)
def test_update_far_from_one_without_eps(rows, cols, scale):
    """fp32's subnormal and largest numbers: the result of the same matrix anywhere else, to the operands' roundings in
    fp16 (as if they fell at other places: twice) and the result's in bfloat16."""
    log("ortho %dx%d times %g" % (rows, cols, scale))
    g = (make((rows, cols), torch.float64, 22).clamp(-3, 3) * scale).float()
    ref = train_ref.newton_schulz(g, 5, eps=0.0)
    held = train_ref.newton_schulz(g, 5, eps=0.0, rounded=True)
    got = gr.orthogonalize(g.cuda(), eps=0.0).cpu().double()
    assert (got - ref).norm() <= 2 * (held - ref).norm() + 2.0 ** -8 * ref.norm()
