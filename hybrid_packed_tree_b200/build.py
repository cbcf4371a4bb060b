"""Build ``libstree.so`` (the C ABI of include/stree.h) in-tree with nvcc for sm_100a, and the
binding's argument check (csrc/bind.cpp) with g++ against the installed torch.

    python -m hybrid_packed_tree_b200.build [--force] [--verbose]

Both are written next to this file so that they travel with the source
tree; nothing is installed into site-packages.  The check's file is named after the torch and
the Python that it was compiled for, and is not needed: where there is none for the present ones
(and no compiler or headers to make it) the binding checks its arguments in Python.
"""
from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libstree.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def bind_path() -> str:
    """Where the argument check for this torch and this Python is, or would be."""
    import torch
    tag = f"{torch.__version__}-abi{int(torch.compiled_with_cxx11_abi())}"
    return os.path.join(PKG, f"_bind.torch-{tag}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_bind(force: bool = False) -> str:
    """Compile csrc/bind.cpp against the installed torch; returns bind_path()."""
    import torch
    bind = bind_path()
    if not force and os.path.exists(bind) and os.path.getmtime(bind) >= os.path.getmtime(BIND_SRC):
        return bind
    at = os.path.dirname(torch.__file__)
    tmp = bind + f".tmp{os.getpid()}"
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                    "-I", sysconfig.get_paths()["include"], "-I", os.path.join(at, "include"),
                    "-I", os.path.join(at, "include", "torch", "csrc", "api", "include"), "-o", tmp, BIND_SRC,
                    "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"], check=True)
    os.replace(tmp, bind)
    return bind


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ into libstree.so, and the argument check; returns the library's path."""
    build_lib(force, verbose)
    try:
        build_bind(force)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"csrc/bind.cpp was not compiled ({e}); arguments are checked in Python, about 3 us a call slower")
    return LIB


def build_lib(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ into libstree.so; returns its path."""
    if not force and not is_stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-lineinfo", "-O3", "-std=c++17",
           "-cudart", "static", "-Xcompiler", "-fPIC", "-shared", "-I", INCLUDE, "-o", tmp, *sources()]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="pass -Xptxas=-v (registers, spills)")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose=args.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
