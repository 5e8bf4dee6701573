"""Build libdsa.so (the C ABI of include/dsa.h) for sm_100a, in-tree, and _dsacall (with the
interpreter's suffix), the extension module through which Python calls it.

The library is one translation unit, csrc/dsa_abi.cu, which includes every
stage's kernels. Compiled with nvcc for sm_100a only. The module
(csrc/dsa_pycall.cpp) is compiled with the C++ compiler against Python's headers, which
must be installed, and linked to the library beside it.
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
LIB = os.path.join(HERE, "libdsa.so")
# Named after the interpreter that it is built for: another one builds its own beside it.
CALL = os.path.join(HERE, "_dsacall" + sysconfig.get_config_var("EXT_SUFFIX"))
CALL_SOURCE = os.path.join(CSRC, "dsa_pycall.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "dsa.h")])


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and os.path.exists(LIB) and all(
            os.path.getmtime(LIB) >= os.path.getmtime(s) for s in sources()):
        build_call(force, verbose)
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *FLAGS, *extra, "-cudart", "static", "-o", tmp, os.path.join(CSRC, "dsa_abi.cu")]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_call(force, verbose)
    return LIB


def build_call(force: bool = False, verbose: bool = False) -> str:
    sources_ = (CALL_SOURCE, os.path.join(ROOT, "include", "dsa.h"))
    if not force and os.path.exists(CALL) and all(
            os.path.getmtime(CALL) >= os.path.getmtime(s) for s in sources_):
        return CALL
    tmp = CALL + f".tmp{os.getpid()}"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-I", sysconfig.get_paths()["include"], "-o", tmp, CALL_SOURCE,
           "-L", HERE, "-l:libdsa.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, CALL)
    return CALL


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "-v" in sys.argv else []))
