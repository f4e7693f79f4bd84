"""Compile the HIP library for gfx950 (``libgemm_relu.so``, in this package) and the
tensor helpers on it (``_tensors.so``, host code on torch's headers, only where
torch is installed).

Run as ``python -m dense_gemm_epilogue_tiled_amd.build``. The library is built
in-tree so the shared object sits next to the Python binding that loads it.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
# one translation unit per family of entry points, compiled side by side
SRC = os.path.join(HERE, "csrc", "gemm_relu.hip")
UNITS = [SRC, os.path.join(HERE, "csrc", "mx_ops.hip")]
LIB = os.path.join(HERE, "libgemm_relu.so")
TENSORS = os.path.join(HERE, "csrc", "tensors.cpp")
EXT = os.path.join(HERE, "_tensors.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # keep the compiler from emitting packed fp32 arithmetic
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    csrc = os.path.join(HERE, "csrc")
    out = [os.path.join(csrc, f) for f in sorted(os.listdir(csrc))]
    out.append(os.path.join(ROOT, "include", "gemm_relu.h"))
    return out


def _run(cmd, verbose, what):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("failed building %s" % what)


def build_tensors(verbose: bool = False) -> str:
    """Build the tensor helpers against the library."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    tmp = EXT + ".tmp%d" % os.getpid()
    try:
        _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
              "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
              "-I", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"],
              "-I", os.path.join(ROOT, "include"), TENSORS, "-L", HERE, "-l:" + os.path.basename(LIB),
              "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
              "-ltorch_hip", "-lc10",
              "-Wl,-rpath,$ORIGIN", "-o", tmp], verbose, EXT)
        os.replace(tmp, EXT)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)
    return EXT


def build(verbose: bool = False) -> str:
    tag = ".tmp%d" % os.getpid()
    objs = [os.path.splitext(u)[0] + tag + ".o" for u in UNITS]
    try:
        jobs = []
        for unit, obj in zip(UNITS, objs):
            cmd = [HIPCC, *FLAGS, "-c", unit, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            jobs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
        outs = [job.communicate()[0] for job in jobs]
        for unit, job, text in zip(UNITS, jobs, outs):
            if job.returncode != 0:
                sys.stderr.write(text)
                raise RuntimeError("hipcc failed compiling %s" % unit)
        _run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", *objs, "-o", LIB + tag], verbose, LIB)
        os.replace(LIB + tag, LIB)
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
    try:
        import torch  # noqa: F401
    except ImportError:
        print("torch is not there: built without the tensor helpers (%s)" % os.path.basename(EXT), flush=True)
        return LIB
    build_tensors(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
