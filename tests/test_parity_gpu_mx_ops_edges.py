"""GPU tests of corners of the operators around the MX products, against the plain fp64 forms (mx_ref)."""
import pytest
import torch

import dense_gemm_epilogue_tiled_amd as gr
import mx_ref
from gpu_util import log
from test_parity_gpu_mx_ops import inputs, weights

pytestmark = pytest.mark.gpu

U = mx_ref.U32


# ---- activations -------------------------------------------------------------------------

def test_silu_far_tail():
    """SiLU below -87, where e^z leaves the normal numbers: 16 roundings as above, at products next to a rounding border."""
    g = torch.arange(-1468, -1400).double().div(16).half()      # -91.75 .. -87.5
    u = (1024 + torch.arange(2048)).half() * 16
    ref = mx_ref.act(g.double(), "silu")[:, None] * u.double()
    y, scale = gr.gated_act(g[:, None].expand(ref.shape).contiguous().cuda(), u.expand(ref.shape).contiguous().cuda(),
                            "silu", "mxfp8")
    mx_ref.check_mx(y.cpu(), scale.cpu(), ref, "mxfp8", 16 * U)


# ---- scales that the conversion cannot apply ----------------------------------------------

@pytest.mark.parametrize("K,waves", [(1024, 8), (8192, 16)])
def test_one_wave_alone_meets_an_unusual_scale(K, waves):
    """Each wave in turn is the only one with a code beyond the conversion (and one turn of units): its products count."""
    M, N = 3, 16
    x = inputs(M, K, "bf16", 200, 2.0 ** 60)
    w, s = weights((N,), K, 201)
    for wave in range(waves):
        log("unusual scale K=%d wave=%d" % (K, wave))
        t = s.clone()
        t[5, K // 32 // waves * wave + 1] = 1
        t[9, K // 32 // waves * wave] = 255
        out = gr.linear_mxfp4(x.cuda(), w.cuda(), t.cuda()).cpu()
        ref, mag = mx_ref.linear(x, w, t)
        assert bool(out[:, 9].isnan().all())
        keep = [n for n in range(N) if n != 9]
        mx_ref.check16(out[:, keep], ref[:, keep], x.dtype, mag[:, keep] * mx_ref.sum_bound(K))


def test_linear_far_scales_cancel_f16():
    """fp16 rows that begin with a small scale: blocks with large ones are finite in fp32 and cancel exactly."""
    M, N, K = 2, 16, 96
    x = torch.zeros(M, K, dtype=torch.float16)
    x[:, 40], x[:, 72] = 1.0, -1.0
    w, s = weights((N,), K, 220)
    w[:, 16:] = 0x22
    s[:, 0], s[:, 1:] = 100, 240
    out = gr.linear_mxfp4(x.cuda(), w.cuda(), s.cuda()).cpu()
    assert bool((out == 0).all()), out


def unusual(s, dtype, seed):
    """Scales with codes in some rows and blocks that the conversion to dtype cannot apply."""
    s = s.clone()
    g = torch.Generator().manual_seed(seed)
    flat = s.view(-1, s.shape[-1])
    rows, blocks = flat.shape
    for r in range(rows):
        b = int(torch.randint(0, blocks, (1,), generator=g))
        if dtype == "f16":  # more than 2^13 apart
            if r % 3 == 0:
                flat[r] = torch.randint(96, 126, (blocks,), generator=g, dtype=torch.uint8)
            elif r % 3 == 1:
                flat[r, b] = 0
        elif r % 2 == 0:
            flat[r, b] = (0, 1, 253, 254)[r // 2 % 4]
    return s


@pytest.mark.parametrize("workspace", ["auto", None])
@pytest.mark.parametrize("M,N,K", [(3, 40, 8736), (16, 50, 16384), (20, 33, 4640), (64, 100, 6176), (64, 16, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_unusual_scales(M, N, K, workspace, dtype):
    """The second go over the units with several passes over K (the sums so far in LDS), with K split over workgroups, and
    with 16 to 64 rows."""
    log("linear unusual M=%d N=%d K=%d dtype=%s workspace=%s" % (M, N, K, dtype, workspace))
    x = inputs(M, K, dtype, 250, 2.0 ** -30 if dtype == "bf16" else 1.0)
    w, s = weights((N,), K, 251)
    s = unusual(s, dtype, 252)
    out = gr.linear_mxfp4(x.cuda(), w.cuda(), s.cuda(), workspace=workspace).cpu()
    ref, mag = mx_ref.linear(x, w, s)
    # products below fp32's normal range are lost: K of them at most
    mx_ref.check16(out, ref, x.dtype, mag * mx_ref.sum_bound(K) + K * 2.0 ** -126)


# ---- experts -------------------------------------------------------------------------------

@pytest.mark.parametrize("I", [64, 1280])
@pytest.mark.parametrize("T", [1, 4, 16])
def test_moe_nan_scale_of_few_tokens(T, I):
    """A NaN scale of one expert stays with the tokens that chose it where all tokens share the second product's tile, in
    one pass over the experts (I = 64) and in two (1280)."""
    log("moe nan scale T=%d I=%d" % (T, I))
    H, E = 128, 4
    x = inputs(T, H, "bf16", 210)
    (w13, s13), (w2, s2) = weights((E, 2 * I), H, 211), weights((E, H), I, 212)
    s2[1, 3, 0] = 255
    ids = torch.tensor([[(t + 1) % 4, 0 if (t + 1) % 4 else 2] for t in range(T)], dtype=torch.int32)
    p = torch.rand(T, 2, generator=torch.Generator().manual_seed(213))
    out = gr.moe_mxfp4(*(t.cuda() for t in (x, ids, p, w13, s13, w2, s2))).cpu()
    want = torch.zeros(T, H, dtype=torch.bool)
    want[(ids == 1).any(1), 3] = True
    assert torch.equal(out.isnan(), want)
    ref, bound = mx_ref.moe(x, ids, p, w13, s13, w2, s2, None, None, "silu")
    zero = torch.zeros(T, H, dtype=torch.float64)
    mx_ref.check16(torch.where(want, zero, out.double()), torch.where(want, zero, ref), x.dtype,
                   torch.where(want, zero, bound))


@pytest.mark.parametrize("T", [2, 20])
def test_moe_hidden_value_beyond_bfloat16(T):
    """h between the products next to fp32's largest value, which bfloat16 rounds to infinity, and infinite itself."""
    log("moe large h T=%d" % T)
    H = I = 32
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[0, 0] = 2.0 ** 60
    w13 = torch.full((1, 2 * I, H // 2), 0x22, dtype=torch.uint8)  # ones
    s13 = torch.full((1, 2 * I, 1), 127 + 4, dtype=torch.uint8)    # g = 2^64
    s13[0, I:] = 127 + 3                                           # u = 2^63
    w2 = torch.full((1, H, I // 2), 0x22, dtype=torch.uint8)
    s2 = torch.full((1, H, 1), 127 - 30, dtype=torch.uint8)
    ids = torch.zeros(T, 1, dtype=torch.int32)
    p = torch.full((T, 1), 2.0 - 2.0 ** -9)                        # h = 1.998 * 2^127
    out = gr.moe_mxfp4(*(t.cuda() for t in (x, ids, p, w13, s13, w2, s2)), act="none").cpu()
    ref, bound = mx_ref.moe(x, ids, p, w13, s13, w2, s2, None, None, "none")
    mx_ref.check16(out, ref, x.dtype, bound)
    s13[0, I:] = 127 + 5                                           # h = 2^129: infinite in fp32
    out = gr.moe_mxfp4(*(t.cuda() for t in (x, ids, p, w13, s13, w2, s2)), act="none").cpu()
    assert bool((out[0] == float("inf")).all()) and bool((out[1:] == 0).all())


@pytest.mark.parametrize("T,H,I,E,k", [(3, 8224, 64, 2, 1), (18, 8224, 64, 2, 1), (18, 32, 4160, 2, 2), (3, 64, 2080, 3, 3),
                                       (5, 96, 160, 4, 2), (40, 256, 512, 3, 2), (1, 64, 96, 4, 2), (12, 4128, 32, 3, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_moe_unusual_scales(T, H, I, E, k, dtype):
    """The second go of the experts' products: pairs of gate and up units, h in two planes, experts side by side in one
    long K (T <= 16) and not, one pass and several. With bfloat16 the second weight has the ends of E8M0 (its products
    are bfloat16 for any x) and small shares keep the sums in range; with fp16 the first one is uneven."""
    log("moe unusual T=%d H=%d I=%d E=%d k=%d dtype=%s" % (T, H, I, E, k, dtype))
    g = torch.Generator().manual_seed(260)
    x = inputs(T, H, dtype, 261)
    (w13, s13), (w2, s2) = weights((E, 2 * I), H, 262, 110, 114), weights((E, H), I, 263)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    p = torch.rand(T, k, generator=g)
    if dtype == "bf16":
        s2, p = unusual(s2, dtype, 264), p * 2.0 ** -40
    else:
        s13 = unusual(s13, dtype, 264)
    out = gr.moe_mxfp4(*(t.cuda() for t in (x, ids, p, w13, s13, w2, s2))).cpu()
    ref, bound = mx_ref.moe(x, ids, p, w13, s13, w2, s2, None, None, "silu")
    mx_ref.check16(out, ref, x.dtype, bound + I * 2.0 ** -126)


def test_moe_most_experts_and_choices():
    """1024 experts and 32 choices: the largest routing tables beside the sums in LDS."""
    for T in (1, 3, 64, 70):
        log("moe most T=%d" % T)
        H, I, E, k = 64, 32, 1024, 32
        g = torch.Generator().manual_seed(270 + T)
        x = inputs(T, H, "bf16", 271)
        (w13, s13), (w2, s2) = weights((E, 2 * I), H, 272), weights((E, H), I, 273)
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
        p = torch.rand(T, k, generator=g)
        out = gr.moe_mxfp4(*(t.cuda() for t in (x, ids, p, w13, s13, w2, s2))).cpu()
        ref, bound = mx_ref.moe(x, ids, p, w13, s13, w2, s2, None, None, "silu")
        mx_ref.check16(out, ref, x.dtype, bound)


@pytest.mark.parametrize("T,H,E,k", [(513, 4096, 64, 8), (1030, 700, 129, 6), (2000, 96, 1000, 20), (5000, 33, 16, 2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_many_tokens(T, H, E, k, renorm):
    """Above 512 tokens one kernel does it: logits within the sums' bounds, weights from them."""
    log("route many T=%d H=%d E=%d k=%d renorm=%s" % (T, H, E, k, renorm))
    x, w = inputs(T, H, "bf16", 280), inputs(E, H, "bf16", 281, 2 * H ** -0.5)
    ids, p = gr.moe_route(x.cuda(), w.cuda(), k, renormalize=renorm)
    ids, p = ids.cpu().long(), p.cpu().double()
    logits = x.double() @ w.double().T
    off = (x.double().abs() @ w.double().abs().T * mx_ref.sum_bound(H)).max().item()
    best = logits.sort(-1, descending=True).values[:, :k]
    top = logits.gather(1, ids)
    assert bool((top - best).abs().max() <= 2 * off) and all(len(set(r)) == k for r in ids.tolist())
    e = torch.exp(top - best[:, :1])
    total = e.sum(-1, keepdim=True) if renorm else torch.exp(logits - best[:, :1]).sum(-1, keepdim=True)
    assert bool(((p - e / total).abs() <= (e / total) * (4 * off + 64 * U)).all())


# ---- MX fp4 x MX fp4 --------------------------------------------------------------------------

def median_us(call, n=15):
    call()
    times = []
    for _ in range(n):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(8):
            call()
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end) / 8 * 1e3)
    return sorted(times)[n // 2]


@pytest.mark.parametrize("M,N,K,streams", [(4096, 4096, 544, False), (8192, 2048, 160, False), (200, 4000, 2080, True),
                                           (300, 300, 8224, True)])
def test_fp4_product_with_ragged_k_takes_the_faster_kernel(M, N, K, streams):
    """Many tiles and a short K go to the guarded kernel (the streaming one takes 3.0 and 2.1 times as long for the first
    two), few tiles or a long K to the streaming one (the guarded one takes 1.9 and 6 times as long). The results are
    right either way."""
    log("fp4 ragged M=%d N=%d K=%d" % (M, N, K))
    (qa, sa), (qb, sb) = weights((M,), K, 230), weights((N,), K, 231)
    dev = [t.cuda() for t in (qa, sa, qb, sb)]
    out = torch.empty(M, N, dtype=torch.float16, device="cuda")
    guarded = median_us(lambda: gr.gemm_mxfp4(*dev, act="none", out=out, path=gr.GR_PATH_TILE_EDGE))
    chosen = median_us(lambda: gr.gemm_mxfp4(*dev, act="none", out=out))
    log("chosen %.1f us, guarded %.1f us" % (chosen, guarded))
    assert chosen < guarded * (0.75 if streams else 1.5)
    a, w = mx_ref.weight(qa[:64], sa[:64]), mx_ref.weight(qb, sb)
    mx_ref.check16(out[:64].cpu(), a @ w.T, torch.float16, (a.abs() @ w.abs().T) * (2.0 ** -16 + mx_ref.sum_bound(K)))


@pytest.mark.parametrize("M,N,K,streams", [(512, 2048, 8192, False), (1024, 1024, 8192, False), (200, 2048, 3584, True),
                                           (16, 8192, 8192, True)])
def test_fp4_product_takes_the_faster_kernel(M, N, K, streams):
    """64 tiles with a long K go to the 128 x 128 tiles (streaming takes 1.4 times as long), fewer rows or a shorter K to
    the streaming kernel (the tiles take 1.2 and 1.6 times as long)."""
    log("fp4 tiles or streaming M=%d N=%d K=%d" % (M, N, K))
    (qa, sa), (qb, sb) = weights((M,), K, 232), weights((N,), K, 233)
    dev = [t.cuda() for t in (qa, sa, qb, sb)]
    out = torch.empty(M, N, dtype=torch.float16, device="cuda")
    tiles = median_us(lambda: gr.gemm_mxfp4(*dev, act="none", out=out, path=gr.GR_PATH_TILE))
    chosen = median_us(lambda: gr.gemm_mxfp4(*dev, act="none", out=out))
    log("chosen %.1f us, tiles %.1f us" % (chosen, tiles))
    assert chosen < tiles * (0.95 if streams else 1.2)


def test_repeated_calls_give_the_same_bits():
    """Sums are added in a fixed order: the same call gives the same bits, one workgroup's K and split ones alike."""
    for M, N, K in ((1, 4096, 4096), (5, 1001, 2080), (64, 1040, 8192)):
        log("repeated M=%d N=%d K=%d" % (M, N, K))
        x = inputs(M, K, "bf16", 240).cuda()
        w, s = (t.cuda() for t in weights((N,), K, 241))
        q, e = gr.mx_quantize(x, "mxfp4")
        first = gr.linear_mxfp4(x, w, s), gr.gemm_mxfp4(q, e, w, s, act="none")
        for _ in range(20):
            again = gr.linear_mxfp4(x, w, s), gr.gemm_mxfp4(q, e, w, s, act="none")
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
