"""Build ``libfp4q.so`` (hand-written HIP for gfx950) in-tree with hipcc, and
``_row_calls.so``, the binding's compiled argument marshalling (host C++).

The library needs hipcc alone (``build_library``, or ``--library`` on the
command line); the marshalling also torch, a host compiler and Python's
headers, as the binding that it belongs to.

Every source is compiled for gfx950 only, with FMA contraction off (the
quantizers' binary32 steps must round exactly as written), packed-fp32
instructions disabled, and HIP's default correctly rounded fp32 division.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
OUT = os.path.join(HERE, "libfp4q.so")
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["matvec_mx.hip", "matvec_nv.hip", "norm_grad.hip", "norm_grad_pack8.hip", "norm.hip", "quant.hip",
           "gemm_mx.hip", "gemm_nv.hip", "swiglu.hip", "swiglu_grad.hip", "dropout.hip", "rotary.hip", "pack8.hip",
           "fp4q_api.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fvisibility=hidden",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-function",
]


ROW_CALLS_OUT = os.path.join(HERE, "_row_calls.so")


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: libfp4q needs ROCm's hipcc to build")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")
    return obj


def _row_calls(verbose: bool) -> None:
    import torch
    from torch.utils import cpp_extension

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    includes = [sysconfig.get_paths()["include"], *cpp_extension.include_paths()]
    tmp = ROW_CALLS_OUT + ".tmp"
    cmd = [_host_compiler(), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in includes),
           os.path.join(CSRC, "row_calls.cpp"), "-o", tmp, f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on row_calls.cpp:\n{r.stderr}")
    os.replace(tmp, ROW_CALLS_OUT)


def _host_compiler() -> str:
    for cand in ("g++", "c++", "clang++", "/opt/rocm/bin/amdclang++"):
        if shutil.which(cand):
            return shutil.which(cand)
    raise RuntimeError("no host C++ compiler found for row_calls.cpp")


def build_library(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(4, len(SOURCES))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = OUT + ".tmp"
    cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, OUT)
    return OUT


def build(verbose: bool = False) -> str:
    """Both. The library is there whatever becomes of the marshalling, which
    is left out where there is no torch, and so no binding, to use it."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        rows = ex.submit(_row_calls, verbose) if importlib.util.find_spec("torch") else None
        out = build_library(verbose)
        if rows is not None:
            rows.result()
        else:
            print(f"torch is not installed: {ROW_CALLS_OUT} is not built", flush=True)
    return out


if __name__ == "__main__":
    print((build_library if "--library" in sys.argv else build)(verbose="-v" in sys.argv))
