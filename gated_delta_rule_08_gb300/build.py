"""Builds libkda.so in-tree with nvcc for sm_103a (no CMake, no torch extension).

Each .cu file under csrc/ is compiled in parallel to an object, then linked into
gated_delta_rule_08_gb300/libkda.so (CUDA runtime linked statically).  Beside it, g++ builds
the Python module that marshals the attention layer's operators, against the installed torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libkda.so")
MARSHAL = os.path.join(PKG, "_kda_marshal.so")
BUILD_DIR = os.path.join(PKG, "_build")
MARSHAL_FOR = os.path.join(BUILD_DIR, "marshal_for")  # what the module has been built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: cannot build libkda.so")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _marshal_command(target: str) -> list:
    import torch
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    includes = [*cpp_extension.include_paths(), sysconfig.get_path("include"), os.path.join(cuda, "include")]
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-I" + i for i in includes),
            os.path.join(CSRC, "kda_marshal.cpp"), *("-L" + p for p in cpp_extension.library_paths()),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-o", target]


def _marshal_stale(deps) -> bool:
    """Whether the marshalling module has to be built: it is bound to torch's C++ interface and to this interpreter's, so it
    is rebuilt when either has been exchanged, whatever the files' times say."""
    return _stale(MARSHAL, deps) or not os.path.exists(MARSHAL_FOR) or open(MARSHAL_FOR).read() != _marshal_for()


def _marshal_for() -> str:
    import torch

    return f"torch {torch.__version__} {os.path.dirname(torch.__file__)}, Python {sys.version}, {platform.machine()}\n"


def build_library(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                     [os.path.join(os.path.dirname(PKG), "include", "kda.h")])
    objs = []
    jobs = []
    for src in sources:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
            if ptxas_v:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    marshal = f"{MARSHAL}.tmp{os.getpid()}"
    remake = force or _marshal_stale([os.path.join(CSRC, "kda_marshal.cpp"), headers[-1]])
    compiled = list(jobs)
    if remake:
        jobs.append(_marshal_command(marshal))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0 or ptxas_v:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {cmd[-1]}")
    if remake:
        os.replace(marshal, MARSHAL)
        with open(MARSHAL_FOR, "w") as f:
            f.write(_marshal_for())
    if force or compiled or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fvisibility=hidden"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of libkda.so failed")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build_library(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_v="--ptxas-v" in sys.argv)
    print(LIB)
