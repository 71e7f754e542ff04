"""Compile libsgemm.so in-tree with nvcc for sm_103a (GB300), and the native part of the
Python binding with the host compiler.

``python -m dense_fp32_matrix_04_gb300.build`` builds them; ``build()`` does the
same from Python and returns the library path.  The ptxas resource report
(registers, spills, shared memory per kernel) is kept in ``_build/ptxas.log``.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libsgemm.so")
NATIVE = os.path.join(PKG, "_native" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILD_DIR = os.path.join(PKG, "_build")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["sgemm_api.cu", "layers_api.cu", "i8_api.cu", "fp4_api.cu", "layer_norm_api.cu", "beam_api.cu"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand) and not shutil.which(cand):
        raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit's bin on PATH")
    return cand


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    files += [os.path.join(ROOT, "include", h) for h in ("sgemm.h", "sgemm_layers.h", "sgemm_layers_testing.h", "sgemm_testing.h")]
    files.append(os.path.abspath(__file__))
    return files


def _torch_dir() -> str | None:
    """Where torch is installed, found without importing it."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _native_command(out: str) -> list[str]:
    """Compiles csrc/native.cpp, which calls libsgemm.so and torch's allocator."""
    torch = _torch_dir()
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include"),
               sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-c", "-o", out,
            *(f for i in include for f in ("-isystem", i)), os.path.join(CSRC, "native.cpp")]


def _native_link(out: str, obj: str) -> list[str]:
    lib = os.path.join(_torch_dir(), "lib")
    return [os.environ.get("CXX") or "g++", "-shared", "-o", out, obj, "-L", PKG, "-l:libsgemm.so", "-L", lib, "-lc10",
            "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or (_torch_dir() and not os.path.exists(NATIVE)):
        return False
    t = min(os.path.getmtime(f) for f in (LIB, NATIVE) if os.path.exists(f))
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
    native = os.path.join(BUILD_DIR, "native.cpp" + tag + ".o") if _torch_dir() else None
    if native:
        jobs.append(_native_command(native))
    with ThreadPoolExecutor(len(jobs)) as pool:
        done = list(pool.map(lambda cmd: subprocess.run(cmd, capture_output=True, text=True), jobs))
    if not any(r.returncode for r in done):
        jobs.append([*common, "-shared", "-o", LIB + tag, *objects])
        done.append(subprocess.run(jobs[-1], capture_output=True, text=True))
    report = "".join(r.stdout + r.stderr for r in done)
    with open(os.path.join(BUILD_DIR, "ptxas.log"), "w") as f:
        f.write("".join(" ".join(cmd) + "\n" for cmd in jobs) + report)
    if native and not any(r.returncode for r in done):
        os.replace(LIB + tag, LIB)
        jobs.append(_native_link(NATIVE + tag, native))
        done.append(subprocess.run(jobs[-1], capture_output=True, text=True))
        report = "".join(r.stdout + r.stderr for r in done)
    for o in objects + [native or ""]:
        if os.path.exists(o):
            os.remove(o)
    if any(r.returncode for r in done):
        sys.stderr.write(report)
        raise RuntimeError(f"nvcc failed; see {BUILD_DIR}/ptxas.log")
    if verbose:
        sys.stdout.write(report)
    os.replace(*((NATIVE + tag, NATIVE) if native else (LIB + tag, LIB)))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
