"""Build libemu_gemm.so in-tree with nvcc for sm_103a (GB300)."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("emu_gemm.cu", "exchange.cu", "experts.cu", "feed_forward.cu", "few_rows.cu", "few_rows_bwd.cu", "few_tiles.cu", "gemm_act.cu", "gemm_gated.cu",
                                              "gemm_gated_bwd.cu", "gemm_rows.cu", "gemm_rows_gated.cu",
                                              "gemm_two.cu", "gemm_two_gated_bwd.cu", "layer_norm.cu", "rms_norm.cu", "route.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("activation.cuh", "aligned.cuh", "emu_kernel.cuh", "few_rows.h", "few_rows_bwd.h", "few_tiles.h", "gemm_epi.h", "group_rows.cuh", "internal.h",
                                                  "norm_rows.cuh",
                                                  "ptx.cuh", "row_ops.cuh")] + [
    os.path.join(os.path.dirname(HERE), "include", "emu_gemm.h")]
LIB = os.path.join(HERE, "libemu_gemm.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libemu_gemm.so")


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in DEPS if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    flags = [ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v" if verbose else "-O3"]
    objects = [f"{tmp}.{os.path.basename(src)}.o" for src in SOURCES]

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)

    try:
        # the files are independent: compiled side by side, then linked
        with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as pool:
            list(pool.map(run, [[nvcc()] + flags + ["-c", "-o", o, src] for src, o in zip(SOURCES, objects)]))
        # The CUDA runtime is linked dynamically, so that a process with PyTorch
        # has one runtime: with a copy of its own in this library, the first
        # call into either after the other cost 2.3 us on a GB300's host.
        lib64 = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "lib64")
        run([nvcc(), ARCH, "-shared", "-cudart", "shared", "-Xlinker", f"-rpath,{lib64}", "-o", tmp] + objects)
        os.replace(tmp, LIB)
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
