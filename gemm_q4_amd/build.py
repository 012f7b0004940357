"""Build libq4_0.so (the HIP kernels and the C ABI) for gfx950 with hipcc, and
_bind.so (the torch conveniences' marshalling, host code) with g++.

Each HIP source compiles to an object under gemm_q4_amd/_build/, in parallel,
then one link step writes gemm_q4_amd/libq4_0.so next to this file.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libq4_0.so")
BIND = os.path.join(HERE, "_bind.so")
CXX = os.environ.get("CXX", "g++")
SOURCES = ["q4_0_api.hip", "q4_0_repack.hip", "q4_0_gemv_dpp.hip",
           "q4_0_gemv_mfma.hip", "q4_0_gemv_w4a8.hip", "q4_0_gemm.hip",
           "q4_0_append.hip", "q4_0_attention.hip", "q4_0_attention8.hip", "q4_0_norm.hip",
           "q4_0_embed.hip", "q4_0_verify.hip", "q4_0_calibrate.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # packed fp32 arithmetic is kept out of the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def _compile(src: str, verbose: bool, build_dir: str = BUILD, extra=()) -> str:
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr.strip():
        print(r.stderr, flush=True)
    return obj


def _build_bind(verbose: bool = False) -> str:
    """Host code against the installed torch (whose libraries are loaded before
    the module is, so it needs no search path for them)."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND + ".tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DQ4_0_TORCH_VERSION="{torch.__version__}"',
           "-I", os.path.join(ROOT, "include"), "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "q4_0_bind.cpp"), "-L", lib, "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed on q4_0_bind.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    return BIND


def build(verbose: bool = False, jobs: int = 8, lib: str = LIB, build_dir: str = BUILD,
          extra=()) -> str:
    """Compile and link; `extra` adds compiler flags (e.g. -D tuning knobs)."""
    os.makedirs(build_dir, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        bind = ex.submit(_build_bind, verbose) if lib == LIB else None
        objs = list(ex.map(lambda s: _compile(s, verbose, build_dir, extra), SOURCES))
        if bind is not None:
            bind.result()
    tmp = lib + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
