"""Build ``libkvattn.so`` in-tree with nvcc for sm_100a, and the binding's ``_marshal.so``.

``python kv_cache_decode_attn_b200/build.py`` (or ``build()``) compiles every
``csrc/*.cu`` and ``csrc/*.cpp`` file into one shared library beside this file.  The library links
the CUDA runtime statically and reaches the driver API (tensor-map encoding)
through ``cudaGetDriverEntryPointByVersion``, so it needs no ``-lcuda`` at link
time.  ``binding/marshal.cpp`` (argument checks of the Python binding, compiled against
the installed torch's headers) becomes ``_marshal.so``, which calls the library beside it.
Rebuilds only when a source is newer than what it makes, and the binding also for another
torch or Python than it was built for: both have C++ and C interfaces of their own.
"""

from __future__ import annotations

import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libkvattn.so")
BINDING = os.path.join(HERE, "binding", "marshal.cpp")
MARSHAL = os.path.join(HERE, "_marshal.so")
MARSHAL_KEY = os.path.join(HERE, "_build", "marshal.key")   # what MARSHAL was built for

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    # CUDA sources and the host-only C++ sources (nvcc hands .cpp files to the host compiler)
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def binding_key() -> str:
    """The torch and Python that a binding built now is for; the package compares it when it is imported."""
    return f"torch {importlib.metadata.version('torch')}, {sysconfig.get_config_var('SOABI')}"


def _binding_stale() -> bool:
    if not os.path.exists(MARSHAL) or not os.path.exists(MARSHAL_KEY):
        return True
    with open(MARSHAL_KEY) as f:
        if f.read() != binding_key():
            return True
    t = os.path.getmtime(MARSHAL)
    return any(os.path.getmtime(p) >= t for p in (BINDING, os.path.join(INCLUDE, "attn.h")))


def build_binding(force: bool = False, verbose: bool = False) -> str:
    if not force and not _binding_stale():
        return MARSHAL
    import torch
    from torch.utils import cpp_extension

    inc = [f"-I{INCLUDE}", f"-isystem{sysconfig.get_paths()['include']}"]
    inc += [f"-isystem{d}" for d in cpp_extension.include_paths()]
    tmp = MARSHAL + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DKVATTN_BUILT_FOR="{binding_key()}"', *inc, BINDING, "-o", tmp,
           f"-L{HERE}", "-l:libkvattn.so", "-Wl,-rpath,$ORIGIN",
           *(f"-L{d}" for d in cpp_extension.library_paths()), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, MARSHAL)
    os.makedirs(os.path.dirname(MARSHAL_KEY), exist_ok=True)
    with open(MARSHAL_KEY, "w") as f:
        f.write(binding_key())
    return MARSHAL


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        build_binding(force, verbose)
        return LIB
    nvcc = _nvcc()
    objs = []
    build_dir = os.path.join(HERE, "_build")
    os.makedirs(build_dir, exist_ok=True)
    for src in sources():
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH_FLAGS, *FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    # export only the C-ABI symbols declared in include/attn.h
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
