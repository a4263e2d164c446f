"""Build the sm_100a shared library ``libsvdq.so`` in-tree with nvcc, and the
compiled binding ``_binding.so`` of the 8-bit and rotary calls above it with the
host compiler.

    python -m bit_quantized_diffusion_b200.build

The library is one translation unit (csrc/svdq.cu) exporting the C ABI of
include/svdq.h. The CUDA runtime is linked statically; the driver's
cuTensorMapEncodeTiled is looked up at run time, so no libcuda is needed at
link time.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libsvdq.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_DEPS = [os.path.join(PKG, "csrc", "binding.cpp"), os.path.join(ROOT, "include", "svdq.h")]
SOURCES = [os.path.join(PKG, "csrc", "svdq.cu")]
DEPS = SOURCES + [os.path.join(PKG, "csrc", f) for f in os.listdir(os.path.join(PKG, "csrc"))
                  if f.endswith(".cuh")] + [os.path.join(ROOT, "include", "svdq.h")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def command(out: str = LIB, verbose_ptxas: bool = False) -> list[str]:
    cmd = [nvcc(), "-shared", "-Xcompiler", "-fPIC", "-O3", "-std=c++17",
           "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
           "-I", os.path.join(ROOT, "include"), "-o", out, *SOURCES]
    if verbose_ptxas:
        cmd[1:1] = ["-Xptxas", "-v"]
    return cmd


def built_for() -> str:
    """What a compiled binding belongs to besides its sources: this interpreter and this torch."""
    import torch
    return (f"{sys.implementation.cache_tag}, torch {torch.__version__}, "
            f"C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}")


def binding_command(out: str = BINDING) -> list[str]:
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no C++ compiler found")
    # libsvdq.so is found beside the binding, so both bindings share one library
    return [cxx, "-shared", "-fPIC", "-O2", "-std=c++17",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DSVDQ_BUILT_FOR="{built_for()}"',
            "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(home, "include"),
            "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), "-o", out, BINDING_DEPS[0],
            "-L", PKG, "-l:libsvdq.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(home, "lib"),
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def up_to_date(out: str = LIB, deps=DEPS) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(d) <= t for d in deps)


def binding_up_to_date(out: str = BINDING, deps=BINDING_DEPS) -> bool:
    """Newer than its sources, and built for the torch that will load it: the module holds the text of
    built_for(). (Another torch's symbols differ, and the import would fail.)"""
    if not up_to_date(out, deps):
        return False
    with open(out, "rb") as f:
        return built_for().encode() + b"\0" in f.read()


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if force or not up_to_date():
        tmp = LIB + ".tmp"
        subprocess.run(command(tmp, verbose_ptxas), check=True)
        os.replace(tmp, LIB)
    if force or not binding_up_to_date():
        tmp = BINDING + ".tmp"
        subprocess.run(binding_command(tmp), check=True)
        os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
    print(LIB)
