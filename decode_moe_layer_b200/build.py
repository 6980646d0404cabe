"""Build libmoe.so (in-tree, next to this file) from csrc/*.cu for sm_100a, and _ops.so, the compiled half of the
Python binding (csrc/python_ops.cpp, plain C++ against torch and libmoe.so).

    python decode_moe_layer_b200/build.py [--force] [--verbose]

(run it by path: importing the package loads the library it builds)

The library links the CUDA runtime statically and reaches the driver's
cuTensorMapEncodeTiled through cudaGetDriverEntryPoint, so it needs no -lcuda.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe.so")
BINDING_SRC = os.path.join(CSRC, "python_ops.cpp")
BINDING = os.path.join(HERE, "_ops.so")
BINDING_KEY = os.path.join(ROOT, "_build", "_ops.key")
CUDA_HOME = os.environ.get("CUDA_HOME", "/usr/local/cuda")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
    "--expt-relaxed-constexpr",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    lib = build_library(force, verbose)
    build_binding(force)
    return lib


def build_binding(force: bool = False) -> str:
    """_ops.so is made for one torch and one Python: besides its sources' times it is kept by a key of the command and of
    their versions, written beside the objects."""
    import torch
    base = os.path.dirname(torch.__file__)
    command = [
        "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-Wall",
        "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi()),
        "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(base, "include"),
        "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
        "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(CUDA_HOME, "include"),
        BINDING_SRC, "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
        "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L", HERE, "-lmoe", "-Wl,-rpath,$ORIGIN"]
    key = "\n".join([torch.__version__, str(sysconfig.get_config_var("SOABI"))] + command)
    deps = [BINDING_SRC, os.path.join(ROOT, "include", "moe.h")]
    if not force and os.path.exists(BINDING) and all(os.path.getmtime(d) <= os.path.getmtime(BINDING) for d in deps):
        try:
            with open(BINDING_KEY) as f:
                if f.read() == key:
                    return BINDING
        except OSError:
            pass
    tmp = BINDING + ".tmp%d" % os.getpid()
    subprocess.check_call(command + ["-o", tmp])
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_KEY), exist_ok=True)
    with open(BINDING_KEY, "w") as f:
        f.write(key)
    return BINDING


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    objdir = os.path.join(ROOT, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [NVCC] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = False
    for cmd, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed = True
            sys.stderr.write(" ".join(cmd) + "\n" + text)
        elif verbose and text:
            sys.stderr.write(text)
    if failed:
        raise RuntimeError("nvcc failed")
    tmp = LIB + ".tmp%d" % os.getpid()
    subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC"]
                          + objs + ["-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
