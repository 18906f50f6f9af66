"""Builds libnvfp4_moe.so in-tree with nvcc for sm_100a (cross-compiles without a GPU), then, if
torch, Python's headers and a host compiler are there, the torch binding of the products' common
calls, which the library does without."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libnvfp4_moe.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-I", INCLUDE]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def marshal_path() -> str:
    """The binding's file for the torch and the Python that run this: it uses both from inside, so
    one built for others is another file."""
    import sysconfig

    import torch
    return os.path.join(HERE, f"_marshal-torch{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_marshal(force: bool = False) -> str:
    """csrc/marshal.cpp against the torch and the Python that run this."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    path, src = marshal_path(), os.path.join(CSRC, "marshal.cpp")
    deps = [src, *glob.glob(os.path.join(INCLUDE, "*.h"))]
    if not force and os.path.exists(path) and os.path.getmtime(path) > max(map(os.path.getmtime, deps)):
        return path
    tmp = path + f".tmp{os.getpid()}"
    includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
                *cpp_extension.include_paths()]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    subprocess.check_call([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in includes],
                           src, "-o", tmp, f"-L{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, jobs: int = 8) -> str:
    """The library; the binding too where it can be built (without it the Python calls take longer)."""
    build_library(force, verbose)
    try:
        build_marshal(force)
    except Exception as e:      # no torch, no Python.h, no compiler, ...
        print(f"warning: the binding of the products' calls was not built ({type(e).__name__}: {e})", file=sys.stderr)
    return LIB


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    procs, objs = [], []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [NVCC, *FLAGS, "-c", src, "-o", obj] + (["-Xptxas", "-v"] if verbose else [])
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode:
            sys.stderr.write(out.decode())
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                           "-o", tmp, *objs, "-lcudart_static", "-lrt",
                           "-ldl", "-lpthread"])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
