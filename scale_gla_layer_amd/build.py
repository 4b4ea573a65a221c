"""Builds libmsgla.so (all HIP kernels + the C ABI) for gfx950 with hipcc.

    python -m scale_gla_layer_amd.build

Objects go to _build/ at the repository root; the shared library is written
next to this file, where the Python binding loads it from.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmsgla.so")
ARCH = os.environ.get("MSGLA_OFFLOAD_ARCH", "gfx950")

SOURCES = [
    "api.cpp",
    "k_pool.hip",
    "k_pool_proj.hip",
    "k_gla_chunk.hip",
    "k_gla_state.hip",
    "k_hold_fuse.hip",
    "k_state.hip",
    "k_decode.hip",
    "k_pack.hip",
    "k_norm.hip",
    "api_noalloc.hip",
    "k_backward.hip",
    "k_bwd_gemm.hip",
    "api_backward.cpp",
    "k_recurrence.hip",
    "api_recurrence.cpp",
    "k_block_select.hip",
    "k_block_attention.hip",
    "k_block_tiles.hip",
    "k_block_grad.hip",
    "api_block.cpp",
    "k_layer_norm.hip",
    "api_layer_norm.cpp",
    "k_linear.hip",
    "api_linear.cpp",
    "k_window.hip",
    "k_window_dq.hip",
    "k_window_few.hip",
    "k_window_grad.hip",
    "api_window.cpp",
]

# rocBLAS: the backward's plain products (weight and input gradients)
LIBS = ["-L/opt/rocm/lib", "-Wl,-rpath,/opt/rocm/lib", "-lrocblas"]

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # keep the compiler from forming packed fp32 ops (v_pk_*_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result",
    "-I", os.path.join(ROOT, "include"),
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libmsgla.so)")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
    cmd = [hipcc(), *FLAGS]
    if src.endswith(".cpp"):
        cmd += ["-x", "hip"]
    cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if "packed-fp32-ops" not in ln]
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n" + "\n".join(msgs))
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs, *LIBS]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
