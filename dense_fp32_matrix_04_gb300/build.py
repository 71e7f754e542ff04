"""Compile libsgemm.so in-tree with nvcc for sm_103a (GB300).

``python -m dense_fp32_matrix_04_gb300.build`` builds it; ``build()`` does the
same from Python and returns the library path.  The ptxas resource report
(registers, spills, shared memory per kernel) is kept in ``_build/ptxas.log``.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libsgemm.so")
BUILD_DIR = os.path.join(PKG, "_build")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["sgemm_api.cu", "layers_api.cu", "i8_api.cu", "fp4_api.cu", "layer_norm_api.cu", "beam_api.cu"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand) and not shutil.which(cand):
        raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit's bin on PATH")
    return cand


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    files += [os.path.join(ROOT, "include", h) for h in ("sgemm.h", "sgemm_layers.h", "sgemm_testing.h")]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    tag = f".tmp{os.getpid()}"
    common = [_nvcc(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xptxas", "-v", "-Xcompiler", "-fPIC,-O2",
              "-I", os.path.join(ROOT, "include")]
    # one object per source, compiled side by side, then one link
    objects = [os.path.join(BUILD_DIR, s + tag + ".o") for s in SOURCES]
    jobs = [[*common, "-c", "-o", o, os.path.join(CSRC, s)] for o, s in zip(objects, SOURCES)]
    with ThreadPoolExecutor(len(jobs)) as pool:
        done = list(pool.map(lambda cmd: subprocess.run(cmd, capture_output=True, text=True), jobs))
    if not any(r.returncode for r in done):
        jobs.append([*common, "-shared", "-o", LIB + tag, *objects])
        done.append(subprocess.run(jobs[-1], capture_output=True, text=True))
    report = "".join(r.stdout + r.stderr for r in done)
    with open(os.path.join(BUILD_DIR, "ptxas.log"), "w") as f:
        f.write("".join(" ".join(cmd) + "\n" for cmd in jobs) + report)
    for o in objects:
        if os.path.exists(o):
            os.remove(o)
    if any(r.returncode for r in done):
        sys.stderr.write(report)
        raise RuntimeError(f"nvcc failed; see {BUILD_DIR}/ptxas.log")
    if verbose:
        sys.stdout.write(report)
    os.replace(LIB + tag, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
