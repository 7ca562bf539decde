"""Build step for the CUDA library (in-tree, sm_103a only).

``build_library()`` compiles ``csrc/sgr_api.cu`` (the projections) and
``csrc/sgr_kv.cu`` (the attention operators), each with the kernels that it
includes, with nvcc side by side, links them into
``_build/libskinny_gemm_residual.so`` next to this file and returns its path.
Rebuilds when any source or public header is newer than the library.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libskinny_gemm_residual.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]
UNITS = ("sgr_api.cu", "sgr_kv.cu")


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def is_stale(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(s) > t for s in sources())


def _run(commands: list[list[str]], verbose: bool) -> None:
    """Run the commands side by side; raise for the first that fails."""
    running = [subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for cmd in commands]
    outputs = [p.communicate()[0] for p in running]
    for cmd, p, out in zip(commands, running, outputs):
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed ({p.returncode}):\n{' '.join(cmd)}\n{out}")
        if verbose:
            print(out)


def build_library(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None,
                  out_path: str = LIB_PATH) -> str:
    """Compile the library if needed; return the .so path."""
    if not force and not is_stale(out_path):
        return out_path
    os.makedirs(os.path.dirname(out_path), exist_ok=True)
    tmp = out_path + f".tmp{os.getpid()}"
    common = [_nvcc(), *(["-Xptxas=-v"] if verbose else []), *ARCH_FLAGS]
    objects = [f"{tmp}.{unit}.o" for unit in UNITS]
    compiles = [[*common, *NVCC_FLAGS, *(extra_flags or []), f"-I{INCLUDE}", "-c", os.path.join(CSRC, unit), "-o", obj]
                for unit, obj in zip(UNITS, objects)]
    try:
        _run(compiles, verbose)
        _run([[*common, "-shared", *objects, "-o", tmp]], False)
    finally:
        for obj in objects:
            if os.path.exists(obj):
                os.remove(obj)
    os.replace(tmp, out_path)
    return out_path


if __name__ == "__main__":
    import sys

    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
