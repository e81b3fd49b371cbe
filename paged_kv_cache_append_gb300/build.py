"""Builds libnk.so in-tree with nvcc for sm_103a, and the CPython module that
marshals arguments for it (``_pyargs`` with the interpreter's ABI tag, gcc).

Each translation unit under ``csrc/`` is compiled in parallel into
``_build/`` and linked into ``paged_kv_cache_append_gb300/libnk.so``; the
CUDA runtime is linked statically, so the library needs only the driver at
run time.  ``python -m paged_kv_cache_append_gb300.build`` runs it.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnk.so")
# One file per interpreter ABI: it is built against one version's headers, and
# another version looks for its own.
PYARGS = os.path.join(PKG, "_pyargs" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libnk")
    return exe


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    deps.append(os.path.join(ROOT, "include", "nk.h"))
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(d) for d in deps) \
            and not extra:
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj


def build_pyargs() -> str:
    """Compiles csrc/pyargs.c against this interpreter's headers; returns its path."""
    src = os.path.join(CSRC, "pyargs.c")
    untagged = os.path.join(PKG, "_pyargs.so")   # any version would load it
    if os.path.exists(untagged):
        os.remove(untagged)
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(ROOT, "include", "nk.h")))
    if os.path.exists(PYARGS) and os.path.getmtime(PYARGS) >= newest:
        return PYARGS
    tmp = PYARGS + ".tmp"
    cmd = ["gcc", "-O2", "-Wall", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"], "-I",
           os.path.join(ROOT, "include"), src, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed for pyargs.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, PYARGS)
    return PYARGS


def objects(extra: list[str] | None = None) -> list[str]:
    """Compiles the CUDA sources whose objects are not up to date; returns all objects' paths."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        return list(ex.map(lambda s: _compile(s, extra or []), srcs))


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compiles every CUDA source and links libnk.so; returns its path."""
    build_pyargs()
    objs = objects(extra)
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])
