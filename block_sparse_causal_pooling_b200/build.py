"""Builds the CUDA library libstem.so in-tree with nvcc, for sm_100a only.

    python -m block_sparse_causal_pooling_b200.build [--force] [--verbose]

Every .cu / .cpp under csrc/ is compiled separately (in parallel) into _build/, then linked
into block_sparse_causal_pooling_b200/libstem.so with the CUDA runtime linked statically.
csrc/python/ becomes the extension module _decode.so (g++, against torch's headers), the native part
of the decode binding, which calls libstem.so beside it. `-Xptxas -v` resource usage is written to _build/ptxas.log.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libstem.so")
BIND = os.path.join(PKG, "_decode.so")
STAMP = os.path.join(BUILD, "_decode.stamp")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-ffp-contract=off",
          "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libstem.so")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose: bool) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_nvcc()] + ARCH + COMMON + ["-c", src, "-o", obj]
    if src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj, r.stderr


def _build_binding(force: bool) -> None:
    import sysconfig

    import torch

    src = os.path.join(CSRC, "python", "decode_bind.cpp")
    troot = os.path.dirname(os.path.abspath(torch.__file__))
    tinc, tlib = os.path.join(troot, "include"), os.path.join(troot, "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    incs = [INCLUDE, tinc, os.path.join(tinc, "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = BIND + ".tmp"
    # (torch's own libraries are in the process before this module is: no run path to them)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for i in incs:
        cmd += ["-I", i]
    cmd += ["-o", tmp, src, "-L", PKG, "-l:libstem.so", "-L", tlib, "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    # what the module was made with and for, wherever the tree lies: another torch or Python has another
    # binary interface
    stamp = "\n".join([torch.__version__, sys.version] + [c.replace(ROOT, "") for c in cmd])
    made = ""
    if os.path.exists(STAMP):
        with open(STAMP) as f:
            made = f.read()
    if not force and made == stamp and not _stale(BIND, [src, os.path.join(INCLUDE, "stem.h"), LIB]):
        return
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for decode_bind.cpp:\n" + r.stderr)
    os.replace(tmp, BIND)
    os.makedirs(BUILD, exist_ok=True)
    with open(STAMP, "w") as f:
        f.write(stamp)


def build(force: bool = False, verbose: bool = False) -> str:
    _build_library(force, verbose)
    _build_binding(force)
    return LIB


def _build_library(force: bool, verbose: bool) -> None:
    srcs = _sources()
    deps = srcs + _headers() + [os.path.abspath(__file__)]
    if not force and not _stale(LIB, deps):
        return
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose), srcs))
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for (obj, log), src in zip(results, srcs):
            f.write(f"== {os.path.basename(src)}\n{log}\n")
    tmp = LIB + ".tmp"
    cmd = [_nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
