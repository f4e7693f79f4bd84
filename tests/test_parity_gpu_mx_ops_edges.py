"""GPU tests of corners of the operators around the MX products, against the plain fp64 forms (mx_ref)."""
import pytest
import torch

import dense_gemm_epilogue_tiled_amd as gr
import mx_ref
from gpu_util import log
from test_parity_gpu_mx_ops import inputs, weights

pytestmark = pytest.mark.gpu

U = mx_ref.U32


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
