"""Build libpd.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ compiles to an object in parallel; the objects link into
paged_kv_split_gb300/libpd.so against the shared CUDA runtime. A rebuild
happens only when a source or header is newer than the library.

csrc/marshal.cpp and csrc/marshal_serve.cpp become the Python modules _marshal.so
and _marshal_serve.so beside it, against the headers of torch and Python. The
binding works without them, its calls take some 10 us longer: where one cannot be
built there is a warning, and one built for another Python or torch is rebuilt,
and not loaded before that.

    python -m paged_kv_split_gb300.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpd.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_ABI = os.path.join(BUILD_DIR, "marshal.abi")  # what _marshal.so was built for
SERVE_SRC = os.path.join(CSRC, "marshal_serve.cpp")
SERVE = os.path.join(PKG, "_marshal_serve.so")
SERVE_ABI = os.path.join(BUILD_DIR, "marshal_serve.abi")

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
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
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


def marshal_abi() -> str:
    """The Python and the torch that _marshal.so depends on."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        torch = re.search(r"__version__ = '([^']*)'", f.read()).group(1)
    return f"{sysconfig.get_config_var('SOABI')} torch {torch}"


def _fits(lib, mark) -> bool:
    try:
        with open(mark) as f:
            return os.path.exists(lib) and f.read() == marshal_abi()
    except (OSError, AttributeError):
        return False


def marshal_fits() -> bool:
    """_marshal.so is there, for this Python and this torch."""
    return _fits(MARSHAL, MARSHAL_ABI)


def serve_fits() -> bool:
    """The same of _marshal_serve.so."""
    return _fits(SERVE, SERVE_ABI)


def _older(path, inputs) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path)
                                           for p in inputs)


def is_stale() -> bool:
    return _older(LIB, _inputs())


def _module_inputs(src):
    return [src, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.h"))


def marshal_is_stale() -> bool:
    return not marshal_fits() or _older(MARSHAL, _module_inputs(MARSHAL_SRC))


def serve_is_stale() -> bool:
    return not serve_fits() or _older(SERVE, _module_inputs(SERVE_SRC))


def _build_module(src, lib, mark) -> bool:
    """Build one module; without it, a warning and False."""
    tmp = lib + f".tmp{os.getpid()}"
    try:
        cmd = ["g++", *marshal_cflags(), "-shared", "-o", tmp, src, "-L", PKG,
               "-l:libpd.so", *marshal_ldflags(), "-Wl,-rpath,$ORIGIN"]
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        why = r.stdout.decode(errors="replace") if r.returncode else None
        abi = marshal_abi()
    except (OSError, AttributeError) as e:  # no g++, no torch
        why = str(e)
    if why is not None:
        if os.path.exists(tmp):
            os.remove(tmp)
        warnings.warn(f"{lib} was not built; calls take longer without it:\n{why}")
        return False
    if os.path.exists(mark):
        os.remove(mark)  # never a module beside another one's mark
    os.replace(tmp, lib)
    with open(mark, "w") as f:
        f.write(abi)
    return True


def _build_modules(force: bool) -> None:
    """Build the stale ones, side by side."""
    stale = [m for m, old in (((MARSHAL_SRC, MARSHAL, MARSHAL_ABI), marshal_is_stale()),
                              ((SERVE_SRC, SERVE, SERVE_ABI), serve_is_stale())) if force or old]
    with ThreadPoolExecutor(2) as pool:
        list(pool.map(lambda m: _build_module(*m), stale))


def _build_lib(verbose_ptxas: bool, quiet: bool) -> None:
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
        raise RuntimeError(f"nvcc failed:\n{msg}")
    tmp = LIB + f".tmp{os.getpid()}"
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(cc)), "lib64")
    subprocess.run([cc, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", f"-rpath,{cuda_lib}",
                    "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = True) -> str:
    if force or is_stale():
        _build_lib(verbose_ptxas, quiet)
    os.makedirs(BUILD_DIR, exist_ok=True)
    _build_modules(force)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv, quiet=False)
    print(LIB)
