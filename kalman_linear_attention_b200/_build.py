"""Compile the CUDA library ``libkla.so`` in-tree for sm_100a with nvcc, and the
CPython extension ``_mixer.so`` that binds the mixer operators."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from importlib import metadata

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(HERE, "libkla.so")
SOURCES = [os.path.join(CSRC, f) for f in ("kla.cu", "kla_host.cu", "kla_gated.cu", "kla_rotary.cu")]
BINDING = os.path.join(HERE, "_mixer.so")
BINDING_SOURCE = os.path.join(CSRC, "kla_binding.cpp")
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "kla_binding.cpp"] + [os.path.join(INCLUDE, "kla.h")]

NVCC_FLAGS = [
    "-O3", "-std=c++17",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "--threads", "0",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-shared",
]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkla.so")
    return cand


def up_to_date() -> bool:
    if not os.path.exists(LIBRARY):
        return False
    t = os.path.getmtime(LIBRARY)
    return all(os.path.getmtime(f) <= t for f in DEPENDS)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build libkla.so and _mixer.so next to this file (each a no-op when it is
    newer than its sources, and _mixer.so for this torch and Python)."""
    build_library(force, verbose)
    build_binding(force)
    return LIBRARY


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIBRARY
    tmp = LIBRARY + ".tmp"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-o", tmp, *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIBRARY)
    return LIBRARY


def built_for() -> str:
    """The torch and Python that _mixer.so is for; what it was built for stands in it."""
    try:
        torch_version = metadata.version("torch")
    except metadata.PackageNotFoundError:  # torch from a source tree
        import torch
        torch_version = torch.__version__
    return f"torch {torch_version}, Python {sys.version_info.major}.{sys.version_info.minor}"


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING):
        return False
    t = os.path.getmtime(BINDING)
    if not all(os.path.getmtime(f) <= t for f in (BINDING_SOURCE, os.path.join(INCLUDE, "kla.h"))):
        return False
    with open(BINDING, "rb") as f:
        return b"\0" + built_for().encode() + b"\0" in f.read()


def build_binding(force: bool = False) -> str:
    """_mixer.so, linked to torch's libraries and to libkla.so beside it."""
    if not force and binding_up_to_date():
        return BINDING
    import torch
    from torch.utils import cpp_extension
    tmp = BINDING + ".tmp"
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    includes = [INCLUDE, *cpp_extension.include_paths(), sysconfig.get_paths()["include"], cuda]
    libraries = [p for p in cpp_extension.library_paths() if os.path.isdir(p)]
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", BINDING_SOURCE,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DKLA_BUILT_FOR="{built_for()}"',
           *[f"-isystem{p}" for p in includes], "-o", tmp, *[f"-L{p}" for p in libraries], f"-L{HERE}",
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-l:libkla.so", "-Wl,-rpath,$ORIGIN"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(force=True, verbose=True))
