"""CPU tests of corners of the training operators' calls."""
import pytest

import dense_gemm_epilogue_tiled_amd as gr
from test_train_ops import BIG, DB, DW, DX, W, gated, gated_bwd

MOST = 1 << 22


def gated_size(M, I, H):
    return gr.gated_linear_workspace_size(M, I, H)


def gated_bwd_size(M, I, H, dx=DX, dw=DW, db=DB):
    return gr.gated_linear_backward_workspace_size(M, I, H, W, max(H, 1), dx, max(H, 1), dw, db)


@pytest.mark.parametrize("M,I,H", [(1, 8, MOST + 1), (8, 8, MOST + 1), (8, 8, (1 << 31) - 1), ((1 << 31) - 1, 8, (1 << 31) - 1)])
def test_size_of_a_gated_layer_that_the_call_refuses(M, I, H):
    """No pitch holds such rows; the bytes of the largest would not fit 63 bits."""
    assert gated(M=M, I=I, H=H) == gr.GR_ERR_TOO_LARGE
    assert gated_size(M, I, H)[0] == gr.GR_ERR_TOO_LARGE


@pytest.mark.parametrize("M,I,H", [(MOST + 1, 24, 50), ((1 << 31) - 1, (1 << 30) - 1, 8), (8, MOST // 2 - 31, 50), (8, MOST // 2, 64)])
def test_size_of_gated_gradients_that_the_call_refuses(M, I, H):
    for dx, dw, db in ((DX, DW, DB), (DX, None, None), (None, DW, None), (None, None, DB)):
        assert gated_bwd(M=M, I=I, H=H, dx=dx, dw=dw, db=db) == gr.GR_ERR_TOO_LARGE
        assert gated_bwd_size(M, I, H, dx, dw, db)[0] == gr.GR_ERR_TOO_LARGE


def test_sizes_at_the_limits():
    """The largest sides that are taken, and empty ones of any length beside them."""
    for M, I, H in ((8, 8, MOST), (0, 8, MOST + 1), (8, 0, MOST + 1)):
        st, n = gated_size(M, I, H)
        assert st == gr.GR_OK and n >= 0
        assert gated(M=M, I=I, H=H, size=BIG << 10) in (gr.GR_OK, gr.GR_ERR_NO_DEVICE) or M * I > 0
    for M, I, H in ((MOST, 24, 50), (8, MOST // 2 - 32, 50), (8, 24, (1 << 31) - 1)):
        st, n = gated_bwd_size(M, I, H)
        assert st == gr.GR_OK and n > 0 and n % 256 == 0
        assert gated_bwd(M=M, I=I, H=H, size=255) == gr.GR_ERR_SCRATCH
