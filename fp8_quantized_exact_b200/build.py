"""Build the sm_100a shared library in-tree with nvcc (no GPU needed), and the
CPython module of the serving calls with the host compiler."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libsage_b200.so")
# with the ABI tag in its name, so that another Python version in the same tree builds and loads its own
SERVING = os.path.join(BUILD, "_sage_serving" + sysconfig.get_config_var("EXT_SUFFIX"))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    """Compile every .cu under csrc/ and link libsage_b200.so (static cudart);
    then the serving module."""
    os.makedirs(BUILD, exist_ok=True)
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if force or _stale(obj, [src] + headers):
            cmd = [NVCC] + NVCC_FLAGS + (extra or []) + ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            subprocess.check_call(cmd)
        objs.append(obj)
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                               "-cudart", "static", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    build_serving(force)
    return LIB


def build_serving(force: bool = False) -> None:
    """Compile the CPython module of the serving calls.  Where the interpreter's
    headers or a C compiler are missing it is left out, with a message: the
    library and the other calls do not need it, and a serving call says so."""
    src = os.path.join(CSRC, "serving_py.c")
    if force or _stale(SERVING, [src, os.path.join(ROOT, "include", "sage_b200.h")]):
        cc, include = os.environ.get("CC", "gcc"), sysconfig.get_paths()["include"]
        if not os.path.exists(os.path.join(include, "Python.h")) or not shutil.which(cc.split()[0]):
            print(f"serving module not built: it needs {os.path.join(include, 'Python.h')} and {cc}", file=sys.stderr)
            return
        tmp = SERVING + f".tmp{os.getpid()}"
        subprocess.check_call(cc.split() + ["-O2", "-std=c11", "-Wall", "-Wextra", "-fPIC", "-shared",
                               "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"), "-I", include, src, "-o",
                               tmp])
        os.replace(tmp, SERVING)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
