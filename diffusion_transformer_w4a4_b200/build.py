"""Build libsvdq.so (the CUDA library behind include/svdq.h) in-tree with nvcc
for sm_100a, and, where torch is installed, _marshal.so (torch tensors to its
arguments) with g++.
Usage: python -m diffusion_transformer_w4a4_b200.build"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsvdq.so")
# the bounds-checked debug variant: same sources with -DSVDQ_DEBUG_BOUNDS
LIB_DEBUG = os.path.join(HERE, "libsvdq_debug.so")
# the Python module that turns torch tensors into the library's arguments
MARSHAL = os.path.join(HERE, "_marshal.so")
MARSHAL_SRC = os.path.join(CSRC, "torch", "marshal.cpp")
MARSHAL_STAMP = os.path.join(HERE, "_build", "marshal.stamp")  # the versions it was compiled against
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(HERE, "..", "include", "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None, debug: bool = False) -> str:
    """Compile libsvdq.so (or, with debug=True, libsvdq_debug.so: every kernel's
    self-addressed global accesses bounds-checked, errors in the status word)."""
    lib = LIB_DEBUG if debug else LIB
    if force or _stale(lib):
        _build_library(lib, verbose, extra, debug)
    if importlib.util.find_spec("torch") is not None:  # the C library does without
        build_marshal(force, verbose)
    return lib


def _build_library(lib: str, verbose: bool, extra: list[str] | None, debug: bool) -> None:
    if debug:
        extra = list(extra or []) + ["-DSVDQ_DEBUG_BOUNDS"]
    nvcc = os.environ.get("NVCC", "nvcc")
    objdir = os.path.join(HERE, "_build_debug" if debug else "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-ffp-contract=off",
               "--fmad=false" if src.endswith("host_prepare.cpp") else "--fmad=true",
               "-I", os.path.join(HERE, "..", "include"), "-c", src, "-o", obj, *(extra or [])]
        if src.endswith(".cpp"):
            cmd = [nvcc, *ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC,-ffp-contract=off,-pthread",
                   "-I", os.path.join(HERE, "..", "include"), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append(subprocess.Popen(cmd))
        objs.append(obj)
    bad = [p.args for p in procs if p.wait() != 0]
    if bad:
        raise RuntimeError(f"nvcc failed for: {[b[-3] for b in bad]}")
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lpthread"])
    os.replace(tmp, lib)


def _marshal_versions() -> str:
    """What _marshal.so is compiled against besides its own source."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # a source tree
        import torch

        version = torch.__version__
    return f"python {sys.version_info[0]}.{sys.version_info[1]} torch {version}"


def _marshal_stale() -> bool:
    header = os.path.join(HERE, "..", "include", "svdq.h")
    if not (os.path.exists(MARSHAL) and os.path.exists(MARSHAL_STAMP)):
        return True
    if any(os.path.getmtime(p) > os.path.getmtime(MARSHAL) for p in (MARSHAL_SRC, header)):
        return True
    with open(MARSHAL_STAMP) as f:
        return f.read() != _marshal_versions()


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """Compile _marshal.so against the installed torch and Python."""
    import sysconfig

    if not force and not _marshal_stale():
        return MARSHAL
    import torch

    root = os.path.dirname(torch.__file__)
    nvcc = shutil.which(os.environ.get("NVCC", "nvcc"))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc))) if nvcc else "/usr/local/cuda"
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DSVDQ_TORCH_VERSION="{torch.__version__}"', "-I", os.path.join(HERE, "..", "include"),
           *(a for d in inc for a in ("-isystem", d)), MARSHAL_SRC, "-o", tmp, "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, MARSHAL)
    os.makedirs(os.path.dirname(MARSHAL_STAMP), exist_ok=True)
    with open(MARSHAL_STAMP, "w") as f:
        f.write(_marshal_versions())
    return MARSHAL


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv))
