"""Compile the HIP library for gfx950 (``libgemm_relu.so``, in this package).

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
        cmd = [HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", *objs, "-o", LIB + tag]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError("hipcc failed linking %s" % LIB)
        os.replace(LIB + tag, LIB)
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
