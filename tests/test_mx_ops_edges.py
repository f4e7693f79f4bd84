"""CPU tests of corners of the operators around the MX products."""
import os
import re

import pytest
import torch

import dense_gemm_epilogue_tiled_amd as gr

CSRC = os.path.join(os.path.dirname(gr.__file__), "csrc")


def test_flag_of_unusual_scales_is_written_by_its_wave_alone():
    """No barrier orders a workgroup's start and its first turn, so a word that one thread clears and any wave sets
    can lose a wave's 1. Each wave writes a word of its own, whatever its value, before the turn's barrier, and
    nothing else writes there: the words hold the waves' flags after the last barrier in any order of the waves."""
    text = open(os.path.join(CSRC, "w4_stream.hpp")).read()
    assert "int again[NW]" in text
    writes = re.findall(r"lds\.again(\[[^\]]*\])?\s*=[^=]\s*([^;]*);", text)
    assert writes == [("[wave]", "bad")]
    at = text.index("lds.again[wave] = bad")
    assert re.match(r"[^;]*;\s*\}?\s*lds_barrier\(\);", text[at:])


# ---- the tensor helpers' checks, called as mx_ops calls them but with CPU tensors, which they refuse last -------------

def helpers():
    if gr.mx_ops._c is None:
        gr.mx_ops._init()
    return gr.mx_ops._c


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def bytes_(*shape):
    return zeros(*shape, dtype=torch.uint8)


def norm(x=None, weight=None, residual=None, code=gr.GR_OUT_16, out=None, scale_out=None, sum_out=None):
    return helpers().rms_norm(zeros(4, 1) if x is None else x, weight, residual, 1e-6, code, out, scale_out, sum_out, 0)


def gated(gate=None, up=None, code=gr.GR_OUT_16, out=None, scale_out=None):
    return helpers().gated_act(zeros(4, 1) if gate is None else gate, up, gr.GR_ACT_SILU, code, out, scale_out, 0)


def linear(x=None, w=None, s=None, bias=None, out=None):
    return helpers().linear_mxfp4(zeros(4, 32) if x is None else x, bytes_(8, 16) if w is None else w,
                                  bytes_(8, 1) if s is None else s, bias, gr.GR_ACT_NONE, out, None, 0)


def fp4(a=None, sa=None, b=None, sb=None, bias=None, out=None):
    return helpers().gemm_mxfp4(bytes_(4, 16) if a is None else a, bytes_(4, 1) if sa is None else sa,
                                bytes_(8, 16) if b is None else b, bytes_(8, 1) if sb is None else sb, bias,
                                gr.GR_ACT_NONE, gr.GR_FMT_BF16, out, -1, 0)


def route(x=None, router=None, bias=None):
    return helpers().moe_route(zeros(4, 1) if x is None else x, zeros(8, 1) if router is None else router, 2, bias, 1,
                               None, 0)


def moe(x=None, p=None, b2=None, out=None):
    return helpers().moe_mxfp4(zeros(4, 32) if x is None else x, zeros(4, 2, dtype=torch.int32),
                               zeros(4, 2, dtype=torch.float32) if p is None else p, bytes_(3, 64, 16), bytes_(3, 64, 1),
                               bytes_(3, 32, 16), bytes_(3, 32, 1), None, b2, gr.GR_ACT_SILU, out, None, 0)


one = zeros(1, 1).expand(4, 1)  # four rows in one element
one8 = bytes_(1, 1).expand(8, 1)

SHARED_ROWS = [(norm, dict(x=one)), (norm, dict(residual=one)), (norm, dict(out=one)),
               (norm, dict(residual=zeros(4, 1), sum_out=one)),
               (norm, dict(x=zeros(4, 32), code=gr.GR_OUT_MXFP8, out=zeros(4, 32, dtype=torch.float8_e4m3fn), scale_out=one8[:4])),
               (gated, dict(gate=one)), (gated, dict(up=one)), (gated, dict(out=one)),
               (linear, dict(s=one8)), (linear, dict(w=bytes_(1, 16).expand(8, 16))),
               (linear, dict(x=zeros(1, 32).expand(4, 32))),
               (linear, dict(w=bytes_(1, 16), s=bytes_(1, 1), out=one)),
               (linear, dict(out=torch.as_strided(zeros(64), (4, 8), (7, 1)))),
               (fp4, dict(sa=one8[:4])), (fp4, dict(sb=one8)), (fp4, dict(b=bytes_(1, 16), sb=bytes_(1, 1), out=one)),
               (route, dict(x=one)), (route, dict(router=zeros(1, 1).expand(8, 1))),
               (moe, dict(x=zeros(1, 32).expand(4, 32))), (moe, dict(out=zeros(1, 32).expand(4, 32)))]


@pytest.mark.parametrize("call,args", SHARED_ROWS, ids=lambda v: v.__name__ if callable(v) else "-".join(v))
def test_rows_that_share_memory_are_refused(call, args):
    """Expanded tensors have a row stride of 0: read as rows one after the other they would go out of their memory."""
    with pytest.raises(ValueError, match="row stride"):
        call(**args)


@pytest.mark.parametrize("call", [norm, gated, linear, fp4, route, moe])
def test_cpu_tensors_are_refused(call):
    with pytest.raises(ValueError, match="GPU"):
        call()


# ---- gradients -----------------------------------------------------------------------------

def wants(*shape, dtype=torch.bfloat16):
    return zeros(*shape, dtype=dtype).requires_grad_()


WANT_GRADIENTS = [(norm, lambda: dict(x=wants(4, 32))), (norm, lambda: dict(weight=wants(1))),
                  (norm, lambda: dict(residual=wants(4, 1))), (norm, lambda: dict(out=wants(4, 1))),
                  (gated, lambda: dict(gate=wants(4, 32))), (gated, lambda: dict(up=wants(4, 1))),
                  (linear, lambda: dict(x=wants(4, 32))), (linear, lambda: dict(bias=wants(8))),
                  (fp4, lambda: dict(bias=wants(8))), (route, lambda: dict(x=wants(4, 1))),
                  (route, lambda: dict(router=wants(8, 1))), (route, lambda: dict(bias=wants(8, dtype=torch.float32))),
                  (moe, lambda: dict(x=wants(4, 32))), (moe, lambda: dict(p=wants(4, 2, dtype=torch.float32))),
                  (moe, lambda: dict(b2=wants(3, 32)))]


@pytest.mark.parametrize("call,args", WANT_GRADIENTS, ids=lambda v: v.__name__ if v in (norm, gated, linear, fp4, route, moe)
                         else "-".join(v()))
def test_gradients_are_refused(call, args):
    """The operators have no gradients: rather than lose one, they refuse a tensor that asks for it. Without recording
    the call goes on (here to the check for a GPU)."""
    with pytest.raises(RuntimeError, match="no gradient"):
        call(**args())
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        call(**args())


def test_forward_gradients_are_refused():
    import torch.autograd.forward_ad as fw
    with fw.dual_level():
        x = fw.make_dual(zeros(4, 32, dtype=torch.float16), zeros(4, 32, dtype=torch.float16))
        with pytest.raises(RuntimeError, match="no gradient"):
            norm(x=x)
        with pytest.raises(RuntimeError, match="no gradient"):
            gated(gate=x)


# ---- first use -------------------------------------------------------------------------------

def test_first_use_is_seen_whole_by_other_threads(monkeypatch):
    """_run takes a set _c for "ready": at no line of _init may it be set before what _run uses beside it."""
    import sys
    ops = gr.mx_ops
    names = ("_c", "_torch", "_FMT", "_raw_stream", "_device")
    for n in names:
        monkeypatch.setattr(ops, n, None)
    seen = []

    def line(frame, event, arg):
        if ops._c is not None:
            seen.append([n for n in names if getattr(ops, n) is None])
        return line

    before = sys.gettrace()
    sys.settrace(lambda frame, event, arg: line if frame.f_code is ops._init.__code__ else None)
    try:
        ops._init()
    finally:
        sys.settrace(before)
    assert seen and not any(seen), seen


# ---- build -----------------------------------------------------------------------------------

@pytest.mark.parametrize("with_torch", [True, False])
def test_the_library_builds_without_torch(monkeypatch, tmp_path, with_torch):
    """The C library and its ctypes binding do without torch, and so does their build; the tensor helpers need it."""
    import sys
    from dense_gemm_epilogue_tiled_amd import build as b
    made = []

    class Job:
        returncode = 0

        def __init__(self, cmd, **kw):
            open(cmd[cmd.index("-o") + 1], "w").close()

        def communicate(self):
            return "", None

    def run(cmd, verbose, what):
        Job(cmd)
        made.append(os.path.basename(what))

    monkeypatch.setattr(b.subprocess, "Popen", Job)
    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "EXT", str(tmp_path / "ext.so"))
    if not with_torch:
        monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert made == (["lib.so", "ext.so"] if with_torch else ["lib.so"])
    assert sorted(os.listdir(tmp_path)) == (["ext.so", "lib.so"] if with_torch else ["lib.so"])
