"""Build step: compile the CUDA library (sm_100a) in-tree.

    python -m approximate_top_selection_b200.build [--force]

Produces approximate_top_selection_b200/libtopk_b200.so from two translation
units, csrc/topk_api.cu (the selections) and csrc/decode_api.cu (cache,
attention and beam search), compiled side by side, and the extension module
_decode_calls.so (the usual calls of the latter without Python in between)
from csrc/decode_calls.cpp; a unit is compiled again only when a file it
includes is newer than its object.
"""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sys
import time

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libtopk_b200.so")
CALLS = os.path.join(PKG, "_decode_calls.so")
CALLS_SRC = os.path.join(PKG, "csrc", "decode_calls.cpp")
UNITS = [os.path.join(PKG, "csrc", "topk_api.cu"), os.path.join(PKG, "csrc", "decode_api.cu")]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.c*")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def stale() -> bool:
    if not os.path.exists(LIB) or _calls_stale():
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def _includes(path: str, seen=None) -> set:
    """`path` and the files it includes by a quoted name, all the way down."""
    seen = set() if seen is None else seen
    path = os.path.normpath(path)
    if path not in seen:
        seen.add(path)
        with open(path) as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M):
                _includes(os.path.join(os.path.dirname(path), name), seen)
    return seen


def _object(unit: str) -> str:
    return os.path.splitext(unit)[0] + ".o"


def _object_stale(unit: str) -> bool:
    obj = _object(unit)
    return not os.path.exists(obj) or any(os.path.getmtime(s) > os.path.getmtime(obj) for s in _includes(unit))


def _calls_stale() -> bool:
    return not os.path.exists(CALLS) or any(os.path.getmtime(s) > os.path.getmtime(CALLS) for s in _includes(CALLS_SRC))


def _calls_command(out: str) -> list:
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), *["-I" + p for p in inc], CALLS_SRC,
            "-o", out, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
            "-L" + os.path.join(cuda, "lib64"), "-lcudart"]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    flags = ["-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC"]
    if verbose:
        flags.insert(0, "-Xptxas=-v")
    running = []
    began = time.time()  # an object is as old as the sources it was started from
    for unit in UNITS:
        if force or _object_stale(unit):
            tmp = _object(unit) + ".tmp%d" % os.getpid()
            running.append((subprocess.Popen([_nvcc(), *flags, "-c", "-o", tmp, unit]), tmp, _object(unit)))
    if force or _calls_stale():
        tmp = CALLS + ".tmp%d" % os.getpid()
        running.append((subprocess.Popen(_calls_command(tmp)), tmp, CALLS))
    failed = [p.args for p, _, _ in running if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, tmp, obj in running:
        os.utime(tmp, (began, began))
        os.replace(tmp, obj)
    tmp = LIB + ".tmp%d" % os.getpid()
    subprocess.check_call([_nvcc(), *ARCH, "-shared", "-o", tmp, *[_object(u) for u in UNITS]])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
