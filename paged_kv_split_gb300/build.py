"""Build libpd.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ compiles to an object in parallel; the objects link into
paged_kv_split_gb300/libpd.so against the shared CUDA runtime; csrc/marshal.cpp
becomes the Python module _marshal.so beside it. A rebuild happens only when a
source or header is newer than the libraries.

    python -m paged_kv_split_gb300.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpd.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = [
    *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
    "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC,
]


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpd.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + [MARSHAL_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def marshal_cflags() -> list:
    """g++ flags that compile csrc/marshal.cpp."""
    inc = os.path.join(_torch_dir(), "include")
    return ["-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
            "-isystem", inc, "-isystem", os.path.join(inc, "torch/csrc/api/include")]


def marshal_ldflags() -> list:
    lib = os.path.join(_torch_dir(), "lib")
    return ["-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{lib}"]


def is_stale() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(MARSHAL)):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    return any(os.path.getmtime(p) > t for p in _inputs())


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = True) -> str:
    if not (force or is_stale()):
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [cc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    marshal_obj = os.path.join(BUILD_DIR, "marshal.cpp.o")
    cmd = ["g++", *marshal_cflags(), "-c", MARSHAL_SRC, "-o", marshal_obj]
    procs.append((MARSHAL_SRC, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif text and (verbose_ptxas or not quiet):
            sys.stdout.write(text)
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"compiling failed:\n{msg}")
    tmp = LIB + f".tmp{os.getpid()}"
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(cc)), "lib64")
    subprocess.run([cc, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", f"-rpath,{cuda_lib}",
                    "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    tmp = MARSHAL + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-shared", "-o", tmp, marshal_obj, "-L", PKG, "-l:libpd.so",
                    *marshal_ldflags(), "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(tmp, MARSHAL)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv, quiet=False)
    print(LIB)
