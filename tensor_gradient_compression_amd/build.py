"""Build libtgrad.so (gfx950) and its torch binding in-tree with hipcc and g++.

Every HIP source under csrc/ is compiled for gfx950 only, without floating-point
contraction (the Adam and weight-update arithmetic keeps its written rounding order)
and without packed-fp32 instructions, then linked into one shared library next to
this file. csrc/binding.cpp, the part of the Python binding that unpacks torch tensors, is
host code against torch's headers and becomes _tgrad_torch.so (left out without torch; the
library itself is a C library and needs hipcc alone).
Usage: python -m tensor_gradient_compression_amd.build
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtgrad.so")
BINDING = os.path.join(PKG, "_tgrad_torch.so")

ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result", "-I", INCLUDE, "-I", CSRC,
]


def _hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain is required to build libtgrad")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *FLAGS, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msgs = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{msgs}")
    if msgs.strip():
        print(msgs, file=sys.stderr)
    return obj


def _torch_dir():
    """torch's folder, or None without torch."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _run(cmd, what: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n" + res.stdout + res.stderr)


def _compile_binding() -> str:
    obj = os.path.join(BUILD, "binding.o")
    inc = os.path.join(_torch_dir(), "include")
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(_hipcc())))
    import torch
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1",
          "-DUSE_ROCM=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", os.path.join(rocm, "include"), "-isystem", sysconfig.get_paths()["include"],
          "-I", INCLUDE, "-Wall", "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ on binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    """Against the libraries that torch has loaded by then, and libtgrad.so beside it."""
    lib = os.path.join(_torch_dir(), "lib")
    tmp = BINDING + ".tmp"
    _run(["g++", "-shared", "-fPIC", "-o", tmp, obj, "-L", PKG, "-l:libtgrad.so", "-L", lib,
          "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN",
          f"-Wl,-rpath,{lib}"], "linking the binding")
    os.replace(tmp, BINDING)


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))
    jobs = min(len(srcs), max(1, min(8, os.cpu_count() or 1)))
    with cf.ThreadPoolExecutor(jobs) as ex:
        bound = ex.submit(_compile_binding) if _torch_dir() else None
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, LIB)
    # the library is there whatever the binding lacks
    if bound is not None:
        _link_binding(bound.result())
    elif verbose:
        print("torch not found: built without the torch binding")
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
