"""Build libfa_b200.so in-tree with nvcc for sm_100a.

    python -m io_aware_exact_35_b200.build [--verbose] [--debug]

The library is one CUDA translation unit (csrc/fa_lib.cu) linked against the
static CUDA runtime; it needs no PyTorch headers.  The output lands in
io_aware_exact_35_b200/lib/ so that it travels with the source tree.  Beside it
goes lib/_fa_native.<Python>.torch-<version>.so, the Python binding of the calls that
are short on the GPU (csrc/fa_binding.cpp, host C++ against PyTorch's headers); its
name says which Python and PyTorch it is for, so that another one does not load it.

``--debug`` builds lib/libfa_b200_debug.so with -DFA_DEBUG: the kernels check
every computed global address and TMA coordinate and record FA_ERR_BOUNDS in
the device error word instead of making a bad access (see sm100.cuh).  Point
FA_B200_LIBRARY at it to run a program against the checked kernels.
"""

from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libfa_b200.so")
DEBUG_LIB = os.path.join(LIBDIR, "libfa_b200_debug.so")

BINDING_SOURCES = [os.path.join(CSRC, "fa_binding.cpp"), os.path.join(ROOT, "include", "fa_b200.h")]

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".cu", ".cuh", ".h"))) + [os.path.join(ROOT, "include", "fa_b200.h")]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(s) <= t for s in sources())


def binding_path() -> str:
    """The native binding of the running Python and PyTorch."""
    import torch
    return os.path.join(LIBDIR, f"_fa_native.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")


def build_binding(force: bool = False) -> str:
    binding = binding_path()
    if not force and os.path.exists(binding) and all(
            os.path.getmtime(s) <= os.path.getmtime(binding) for s in BINDING_SOURCES):
        return binding
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    os.makedirs(LIBDIR, exist_ok=True)
    tmp = binding + ".tmp"
    # the system's compiler: one that links its C++ runtime in statically gives the
    # process a second one beside PyTorch's
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in (os.path.join(root, "include"),
                                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                                os.path.join(cuda, "include"), sysconfig.get_paths()["include"])),
           BINDING_SOURCES[0], "-o", tmp, f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("the C++ compiler failed to build the native binding")
    os.replace(tmp, binding)
    return binding


def build(verbose: bool = False, force: bool = False, debug: bool = False) -> str:
    build_binding(force)
    lib = DEBUG_LIB if debug else LIB
    if not force and up_to_date(lib):
        return lib
    os.makedirs(LIBDIR, exist_ok=True)
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH_FLAGS, "-O3", "-std=c++17", "-lineinfo", "--use_fast_math",
           "-Xcompiler", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"),
           *(["-DFA_DEBUG"] if debug else []),
           os.path.join(CSRC, "fa_lib.cu"), "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"nvcc failed to build {os.path.basename(lib)}")
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--debug", action="store_true")
    a = ap.parse_args()
    print(build(verbose=a.verbose, force=a.force, debug=a.debug))
