"""Build ``libokv.so`` in-tree with nvcc for sm_100a (no JIT cache, no torch extension).

Usage: ``python -m int2_kv_cache_rotate_b200.build [--verbose-ptxas] [--short-wait]``.
``--short-wait`` builds the test library ``libokv_shortwait.so`` instead: every
bounded wait of the kernels gives up after 64 cycles (the waits of the timeout
paths for work already issued keep their full limit), so that a test can run
the timeout paths.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libokv.so")
SHORT_WAIT_LIB = os.path.join(HERE, "libokv_shortwait.so")
SOURCES = ["okv_api.cu", "append.cu", "decode.cu", "decode_int4.cu", "dequant.cu", "prefill.cu", "prefill_int4.cu", "prefill_rotate.cu",
           "noalloc.cu", "plan.cu", "norm_rope.cu", "calib.cpp", "rotio.cpp"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def build(verbose_ptxas: bool = False, out: str = LIB, short_wait: bool = False) -> str:
    defs = ["-DOKV_WAIT_LIMIT_LOG2=6"] if short_wait else []
    flags = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", *defs, "-Xcompiler", "-fPIC,-fopenmp,-O3",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if verbose_ptxas:
        flags.insert(1, "-Xptxas=-v")

    def run(cmd):
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
        return res.stderr

    with tempfile.TemporaryDirectory() as tmp:  # one object per source, compiled side by side, then linked
        objs = [os.path.join(tmp, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            logs = list(pool.map(lambda so: run([*flags, "-c", os.path.join(CSRC, so[0]), "-o", so[1]]),
                                 zip(SOURCES, objs)))
        run([nvcc(), *ARCH, "-shared", "-o", out, *objs, "-lgomp"])
    if verbose_ptxas:
        sys.stderr.write("".join(logs))
    return out


if __name__ == "__main__":
    if "--short-wait" in sys.argv:
        print(build(verbose_ptxas="--verbose-ptxas" in sys.argv, out=SHORT_WAIT_LIB, short_wait=True))
    else:
        print(build(verbose_ptxas="--verbose-ptxas" in sys.argv))
