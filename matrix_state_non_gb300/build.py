"""Builds libm2rnn.so in-tree with nvcc for sm_103a (no CMake).

Each CUDA translation unit compiles in parallel, then one link step makes the
shared library next to this file.  Run as ``python -m matrix_state_non_gb300.build``
or through ``__graft_entry__.build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libm2rnn.so")
SOURCES = ["api.cu", "simt.cu", "tc_forward.cu", "tc_backward.cu", "tc_backward128.cu", "mma_forward.cu",
           "mma_backward.cu", "host_util.cu", "noalloc.cu", "decode.cu",
           "mv_forward.cu", "mv_backward.cu", "mv_backward_pipe.cu", "mv_forward_pipe.cu", "gate_norm.cu",
           "layer_api.cu", "conv.cu", "ssm.cu", "ssm_f32.cu", "ssm_mma.cu", "ssm_tc.cu", "ssm_tc_walk.cu",
           "ssm_grad.cu", "grad_clip.cu", "around_api.cu", "residual_norm.cu", "linear_scan.cu", "ortho.cu", "ortho_small.cu", "ortho_thin.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libm2rnn.so")
    return cand


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    extra = list(extra or [])
    if verbose:
        extra += ["-Xptxas", "-v"]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
