"""Build the in-tree CUDA libraries for sm_100a with nvcc.

    python -m fp4_routed_expert_router_b200.build [--force]

Produces lib/libmoe_fp4.so (the compute path, C ABI of include/moe_fp4.h) and
lib/libmoe_synth.so (device-side synthetic-input generator).  nvcc
cross-compiles without a GPU.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]

TARGETS = {
    "libmoe_fp4.so": ["moe_fp4_api.cu", "linear_fwd.cu", "linear_swiglu.cu", "linear_dgrad.cu", "linear_wgrad.cu"],
    "libmoe_synth.so": ["synth_fill.cu"],
}


def _deps() -> list[str]:
    return glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _nvcc(args: list[str]) -> str:
    res = subprocess.run([NVCC, *ARCH, *FLAGS, *args], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc {' '.join(args)} failed\n{res.stdout}{res.stderr}")
    return res.stderr


def build(force: bool = False, verbose: bool = False) -> dict:
    """Compile the sources of every target side by side and link each into its library."""
    os.makedirs(LIBDIR, exist_ok=True)
    newest = max(os.path.getmtime(p) for p in _deps())
    out = {lib: os.path.join(LIBDIR, lib) for lib in TARGETS}
    stale = [lib for lib, dst in out.items()
             if force or not os.path.exists(dst) or os.path.getmtime(dst) < newest]
    if not stale:
        return out
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor() as pool:
        logs = {}
        for lib in stale:
            for src in TARGETS[lib]:
                obj = os.path.join(tmp, f"{lib}.{src}.o")
                logs[obj] = pool.submit(_nvcc, ["-c", os.path.join(CSRC, src), "-o", obj])
        text = "".join(f.result() for f in logs.values())
        for lib in stale:
            objs = [os.path.join(tmp, f"{lib}.{src}.o") for src in TARGETS[lib]]
            new = out[lib] + ".new"
            text += _nvcc(["-shared", *objs, "-o", new])
            os.replace(new, out[lib])
    if verbose:
        sys.stderr.write(text)
    return out


if __name__ == "__main__":
    for k, v in build(force="--force" in sys.argv, verbose="-v" in sys.argv).items():
        print(k, v)
