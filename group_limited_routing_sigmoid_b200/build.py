"""Build ``libbeam_moe.so`` in-tree with nvcc for sm_100a (B200).

    python -m group_limited_routing_sigmoid_b200.build [--force] [--verbose-ptxas]

Each ``csrc/*.cu`` is compiled to an object under ``_build/`` (repo root) and
linked, with the CUDA runtime statically, into
``group_limited_routing_sigmoid_b200/libbeam_moe.so``.  Objects are rebuilt
when their source or any header is newer.  ``csrc/ops_binding.cpp``, the Python
side of ``ops.py``, becomes ``_ops_binding.so`` beside it, with the host
compiler against the installed PyTorch.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libbeam_moe.so")
OPS_BINDING = os.path.join(PKG, "_ops_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest(paths):
    return max(os.path.getmtime(p) for p in paths)


def build_binding(force: bool = False, quiet: bool = False) -> str:
    import torch    # its headers and libraries are compiled against

    src = os.path.join(CSRC, "ops_binding.cpp")
    stamp = os.path.join(BUILD, "ops_binding.torch")   # the version it was compiled against
    known = os.path.exists(stamp) and open(stamp).read() == torch.__version__
    if not force and known and os.path.exists(OPS_BINDING) and \
            os.path.getmtime(OPS_BINDING) >= max(os.path.getmtime(src), _newest(glob.glob(os.path.join(INCLUDE, "*.h")))):
        return OPS_BINDING
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = OPS_BINDING + f".tmp{os.getpid()}"
    # the system's compiler: one that links its own libstdc++ statically would
    # not catch PyTorch's exceptions
    cmd = [shutil.which("g++") or os.environ.get("CXX", "c++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", os.path.join(root, "include"), "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), "-o", tmp, src,
           "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python"]
    if not quiet:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, OPS_BINDING)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return OPS_BINDING


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    hdr_time = _newest(headers) if headers else 0
    objs, commands = [], []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or verbose_ptxas or not os.path.exists(obj) or \
                os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time):
            cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
            if verbose_ptxas:
                cmd += ["-Xptxas", "-v"]
            if not quiet:
                print(" ".join(cmd), flush=True)
            commands.append(cmd)
    with ThreadPoolExecutor(max(1, os.cpu_count() or 1)) as pool:   # the sources are independent
        list(pool.map(subprocess.check_call, commands))
    if commands or force or not os.path.exists(LIB) or os.path.getmtime(LIB) < _newest(objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        if not quiet:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    build_binding(force, quiet)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))
    sys.exit(0)
