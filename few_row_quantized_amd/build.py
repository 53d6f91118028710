"""Build libqgemv.so in-tree with hipcc for gfx950, and the Python module
_qgemv_torch.so (its calls on torch tensors) with the host compiler, where torch
and such a compiler are there.

    python -m few_row_quantized_amd.build [-v]

Compiles every source under csrc/ to an object in _build/ (in parallel) and
links few_row_quantized_amd/libqgemv.so.  Always recompiles (the build check
must exercise the compiler every time).
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig
import time

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libqgemv.so")
MODULE = os.path.join(PKG, "_qgemv_torch.so")
ARCH = "gfx950"

COMMON_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-Wall", "-Wno-unused-result",
    # keep hipcc from forming packed-fp32 instructions (v_pk_*_f32) on its own
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]

# the products, and the verify step's other operators
PRODUCTS = ["qgemv_api.cpp", "qgemv_dot.hip", "qgemv_dot_add.hip", "qgemv_dot8.hip", "qgemv_dot_fp.hip",
            "qgemv_mfma.hip",
            "qgemv_persist.hip", "qgemv_persist_x.hip", "qgemv_gather.hip", "qgemv_probe.hip"]
VERIFY_STEP = ["qgemv_kv_api.cpp", "qgemv_append.hip", "qgemv_attend.hip", "qgemv_attend_bf16.hip",
               "qgemv_attend_f16.hip", "qgemv_attend_bf16_e4m3.hip", "qgemv_attend_f16_e4m3.hip", "qgemv_verify.hip",
               "qgemv_prefix_bf16.hip", "qgemv_prefix_f16.hip", "qgemv_prefix_bf16_e4m3.hip",
               "qgemv_prefix_f16_e4m3.hip", "qgemv_route.hip", "qgemv_adapt.hip"]
SOURCES = PRODUCTS + VERIFY_STEP


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libqgemv.so)")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc(), *COMMON_FLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    t0 = time.time()
    proc = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature; drop that line
    err = "\n".join(l for l in proc.stderr.splitlines() if "packed-fp32-ops" not in l)
    if proc.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{err}")
    if verbose:
        print(f"  {src}: {time.time() - t0:.1f}s", flush=True)
        if err.strip():
            print(err)
    return obj


def _module(verbose: bool) -> None:
    """qgemv_torch.cpp: host code alone, against torch's headers.  Where those or
    the host compiler are missing there is no module, and none of an earlier
    build stays; the C library does not need it."""
    cxx = os.environ.get("CXX", "g++")
    try:
        import torch
        root = os.path.dirname(torch.__file__)
    except ImportError:
        root = None
    include = [os.path.join(root or "", "include"),
               os.path.join(root or "", "include", "torch", "csrc", "api", "include")]
    missing = ("torch" if root is None else "torch's headers" if not os.path.isdir(include[0])
               else cxx if shutil.which(cxx.split()[0]) is None else None)
    if missing:
        if os.path.exists(MODULE):
            os.remove(MODULE)
        print(f"  _qgemv_torch not built: {missing} not found (the C library does without; "
              "the verify step's Python calls need it)", flush=True)
        return
    tmp = MODULE + ".tmp"
    cmd = [*cxx.split(), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include"),
           "-I", sysconfig.get_paths()["include"], *(f for i in include for f in ("-isystem", i)),
           os.path.join(CSRC, "qgemv_torch.cpp"), "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    t0 = time.time()
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{proc.stderr}")
    os.replace(tmp, MODULE)
    if verbose:
        print(f"  qgemv_torch.cpp: {time.time() - t0:.1f}s\n{proc.stderr}", end="", flush=True)


def _link(objs) -> None:
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{proc.stderr}")
    os.replace(tmp, LIB)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    t0 = time.time()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        module = ex.submit(_module, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        _link(objs)
        if verbose:
            print(f"built {LIB} in {time.time() - t0:.1f}s", flush=True)
        module.result()  # what failed there, with the library in place
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
