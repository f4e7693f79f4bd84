"""CPU tests: the tensor helpers of the products refuse operands whose rows share memory."""
import pytest
import torch

import dense_gemm_epilogue_tiled_amd as gr

H, B8 = torch.float16, torch.uint8
E4 = torch.float8_e4m3fn


def z(*shape, dtype=H):
    return torch.zeros(*shape, dtype=dtype)


def one(n, dtype=H):
    return z(1, 1, dtype=dtype).expand(n, 1)  # n rows in one element


# each operand in turn with one column and a row stride of 0 (the helpers are given a stream handle, as without a GPU
# there is no current stream; a call that came through would end with GR_ERR_NO_DEVICE)
CASES = {
    "gemm_relu_bt a": lambda: gr.gemm_relu_bt(one(4), z(3, 1), stream=0),
    "gemm_relu_bt bt": lambda: gr.gemm_relu_bt(z(4, 1), one(3), stream=0),
    "gemm_relu_bt out": lambda: gr.gemm_relu_bt(z(4, 5), z(1, 5), out=one(4), stream=0),
    "gemm_relu a": lambda: gr.gemm_relu(one(4), z(1, 3), workspace=None, stream=0),
    "gemm_relu b": lambda: gr.gemm_relu(z(4, 5), one(5), workspace=None, stream=0),
    "gemm_relu out": lambda: gr.gemm_relu(z(4, 5), z(5, 1), out=one(4), workspace=None, stream=0),
    "gemm_bias_act a": lambda: gr.gemm_bias_act(one(4), z(1, 3), workspace=None, stream=0),
    "gemm_bias_act b": lambda: gr.gemm_bias_act(z(4, 5), one(5), workspace=None, stream=0),
    "gemm_bias_act out": lambda: gr.gemm_bias_act(z(4, 5), z(5, 1), out=one(4), workspace=None, stream=0),
    "gemm_fp8 a": lambda: gr.gemm_fp8(one(4, E4), z(3, 1, dtype=E4), workspace=None, stream=0),
    "gemm_fp8 bt": lambda: gr.gemm_fp8(z(4, 1, dtype=E4), one(3, E4), workspace=None, stream=0),
    "gemm_fp8 out": lambda: gr.gemm_fp8(z(4, 5, dtype=E4), z(1, 5, dtype=E4), out=one(4), workspace=None, stream=0),
    "gemm_mxfp8 scale_a": lambda: gr.gemm_mxfp8(z(4, 32, dtype=E4), one(4, B8), z(3, 32, dtype=E4),
                                                z(3, 1, dtype=B8), stream=0),
    "gemm_mxfp8 scale_b": lambda: gr.gemm_mxfp8(z(4, 32, dtype=E4), z(4, 1, dtype=B8), z(3, 32, dtype=E4),
                                                one(3, B8), stream=0),
    "gemm_mxfp8 out": lambda: gr.gemm_mxfp8(z(4, 32, dtype=E4), z(4, 1, dtype=B8), z(1, 32, dtype=E4),
                                            z(1, 1, dtype=B8), out=one(4), stream=0),
    "linear x": lambda: gr.linear(one(4), z(3, 1), stream=0),
    "linear weight": lambda: gr.linear(z(4, 1), one(3), stream=0),
    "linear out": lambda: gr.linear(z(4, 5), z(1, 5), out=one(4), stream=0),
}


@pytest.mark.parametrize("name", CASES)
def test_rows_that_share_memory_are_refused(name):
    with pytest.raises(gr.GemmReluError) as e:
        CASES[name]()
    assert e.value.status == gr.GR_ERR_INVALID_LD


@pytest.mark.parametrize("shape", [(3, 5), (4, 4), (1, 1), (20,)])
@pytest.mark.parametrize("name,call", [
    ("gemm_relu_bt", lambda out: gr.gemm_relu_bt(z(4, 8), z(5, 8), out=out, stream=0)),
    ("gemm_relu", lambda out: gr.gemm_relu(z(4, 8), z(8, 5), out=out, workspace=None, stream=0)),
    ("gemm_bias_act", lambda out: gr.gemm_bias_act(z(4, 8), z(8, 5), out=out, workspace=None, stream=0)),
    ("gemm_fp8", lambda out: gr.gemm_fp8(z(4, 8, dtype=E4), z(5, 8, dtype=E4), out=out, workspace=None, stream=0)),
    ("gemm_mxfp8", lambda out: gr.gemm_mxfp8(z(4, 32, dtype=E4), z(4, 1, dtype=B8), z(5, 32, dtype=E4),
                                             z(5, 1, dtype=B8), out=out, stream=0)),
    ("linear", lambda out: gr.linear(z(4, 8), z(5, 8), out=out, stream=0))], ids=lambda v: v if isinstance(v, str) else "")
def test_output_too_small_is_refused(name, call, shape):
    """A 4 x 5 product does not go into fewer rows or columns."""
    with pytest.raises(ValueError, match="out"):
        call(z(*shape))
