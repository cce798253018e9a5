"""Build the in-tree CUDA library libgemm_f16.so for sm_103a with nvcc.

One object per source (compiled in parallel), one -gencode target,
position-independent, static CUDA runtime.  Rebuilt only when a source or header
is newer than the library.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libgemm_f16.so")
SOURCES = [os.path.join(HERE, "csrc", n) for n in ("gemm_f16.cu", "gemm_mxf4.cu", "moe_f16.cu", "gemm_fp8.cu", "rms_norm.cu",
                                                    "moe_route.cu")]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-I" + os.path.join(ROOT, "include"),
]


def _inputs():
    return (SOURCES + glob.glob(os.path.join(HERE, "csrc", "*.cuh")) + glob.glob(os.path.join(HERE, "csrc", "*.h"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = NVCC if os.path.exists(NVCC) else "nvcc"
    tmp = LIB + f".tmp{os.getpid()}"
    objects = [f"{tmp}.{os.path.basename(s)}.o" for s in SOURCES]
    cmds = [[nvcc, *FLAGS, *extra_flags, "-c", "-o", o, s] for o, s in zip(objects, SOURCES)]
    cmds.append([nvcc, *FLAGS, *extra_flags, "-shared", "-o", tmp, *objects])
    if verbose:
        print("\n".join(" ".join(c) for c in cmds), file=sys.stderr)
    try:
        running = [subprocess.Popen(c) for c in cmds[:-1]]
        codes = [p.wait() for p in running]
        for c, code in zip(cmds, codes):
            if code:
                raise subprocess.CalledProcessError(code, c)
        subprocess.run(cmds[-1], check=True)
        os.replace(tmp, LIB)
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
