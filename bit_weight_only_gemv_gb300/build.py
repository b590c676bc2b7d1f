"""Build the C-ABI library in-tree: bit_weight_only_gemv_gb300/libw4a16.so.

Every CUDA source is compiled for sm_103a only (one -gencode), in parallel,
then linked with the static CUDA runtime.  Usage: ``python -m
bit_weight_only_gemv_gb300.build [--verbose-ptxas]``.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libw4a16.so")
SOURCES = ["gemv.cu", "chain.cu", "gemv_tc.cu", "gemm_tc.cu", "gather.cu", "quant.cu",
           "slot_pool.cu", "dev_pool.cu", "kv8_append.cu", "kv8_select.cu", "kv8_attn.cu",
           "kv8_chunk.cu", "kv8_weigh.cu", "kv8_weigh_tc.cu", "kv8_pages.cu", "route.cu",
           "logits.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose_ptxas:
        cmd[1:1] = ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas:
        sys.stderr.write(res.stderr)
    return obj


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    deps = srcs + [os.path.join(CSRC, "common.cuh"), os.path.join(CSRC, "gemv_core.cuh"),
                   os.path.join(CSRC, "gemv_host.h"), os.path.join(CSRC, "gemv_tc.h"),
                   os.path.join(CSRC, "tc_common.cuh"), os.path.join(CSRC, "pointer_view.h"),
                   os.path.join(CSRC, "kv8.cuh"), os.path.join(CSRC, "kv8_mma.cuh"),
                   os.path.join(CSRC, "kv8_attn.h"), os.path.join(CSRC, "kv8_runs.cuh"),
                   os.path.join(CSRC, "kv8_tc.cuh"),
                   os.path.join(os.path.dirname(PKG), "include", "w4a16.h")]
    if not force and os.path.exists(LIB):
        newest = max(os.path.getmtime(d) for d in deps)
        if os.path.getmtime(LIB) >= newest and not verbose_ptxas:
            return LIB
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose_ptxas="--verbose-ptxas" in sys.argv, force=True))
