"""Build libflce.so (the C-ABI library) in-tree for sm_103a.

The translation units compile in parallel with nvcc and link into one shared
library with a static CUDA runtime, so loading it needs no driver library until the
first CUDA call. Run ``python -m linear_cross_entropy_tcgen05_gb300.build``, optionally
with ``-DNAME=VALUE`` compile-time tunables.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libflce.so")

SOURCES = ["flce_gemm.cu", "flce_small.cu", "flce_api.cu", "flce_noalloc.cu", "flce_block_norm.cu", "flce_grad_clip.cu",
           "flce_beam.cu"]
# the block norm's kernels, one file for each pair of activation and residual types and direction
SOURCES += [f"block_norm_{d}_{t}.cu" for d in ("backward", "forward")
            for t in ("bf16_bf16", "bf16_f32", "f16_f16", "f16_f32", "f32_f32")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libflce.so")
    return exe


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile every translation unit and link libflce.so; returns its path."""
    extra = list(extra or [])
    if verbose:
        extra += ["-Xptxas", "-v"]
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    # python -m linear_cross_entropy_tcgen05_gb300.build [-v] [-DNAME=VALUE ...]
    # -D sets a compile-time tunable of the kernels (e.g. -DFLCE_FWD_PANEL=4).
    defines = [a for a in sys.argv[1:] if a.startswith("-D")]
    print(build(verbose="-v" in sys.argv, extra=defines))
