"""Build libmoe.so (the C-ABI library) in-tree with nvcc for sm_100a, and _ops16.so, its torch binding.

Each .cu file compiles to its own object in _build/ (in parallel, and only when
it or a header changed), then one link step writes libmoe.so next to this file.
csrc/binding.cpp (the 16-bit expert operators on torch tensors) compiles against
torch's headers and links against libmoe.so.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(ROOT, "_build", "moe")
LIB = os.path.join(PKG, "libmoe.so")
BINDING = os.path.join(PKG, "_ops16.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr", "-Xcompiler", "-Wall"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _inputs():
    return sources() + _headers()


def _older(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in inputs)


def _binding_inputs():
    return [BINDING_SRC, os.path.join(INCLUDE, "moe.h")]


def stale() -> bool:
    return _older(LIB, _inputs()) or _older(BINDING, _binding_inputs())


def _build_binding(verbose: bool) -> None:
    import torch
    troot = os.path.dirname(torch.__file__)
    tmp = BINDING + f".tmp{os.getpid()}"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(NVCC)))
    cmd = ["g++", "-O2", "-shared", "-fPIC", "-std=c++17", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", os.path.join(troot, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp, "-L", PKG, "-l:libmoe.so",
           "-Wl,-rpath,$ORIGIN", "-L", os.path.join(troot, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, BINDING)


def _obj(src: str) -> str:
    return os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")


def _compile(src: str, force: bool, ptxas_v: bool, verbose: bool) -> str:
    out = _obj(src)
    newest = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in _headers()])
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest:
        return out
    tmp = out + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", tmp]
    if ptxas_v:
        cmd.insert(1, "-Xptxas=-v")
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    if not force and not stale():
        return LIB
    if not force and not _older(LIB, _inputs()):
        _build_binding(verbose)
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(s, force, ptxas_v, verbose), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    if force or _older(BINDING, _binding_inputs()):
        _build_binding(verbose)
    return LIB


if __name__ == "__main__":
    build(force="-f" in sys.argv, verbose=True, ptxas_v="-v" in sys.argv)
    print(LIB)
