"""Builds libmuon.so in-tree with nvcc for sm_103a (GB300).

Each CUDA translation unit is compiled in parallel into ``_build/`` and the
objects are linked into ``newton_schulz_fp32_gb300/libmuon.so`` (static CUDA
runtime; the driver API is reached through the runtime's entry-point query,
so the library links no libcuda).  A rebuild happens only when a source or
header is newer than the library.  The C half of the Python binding
(``csrc/binding.c``) is compiled with gcc into ``_binding`` plus the interpreter's suffix
beside it, where Python's headers are there; without them the embedding and
loss calls raise and everything else works.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmuon.so")
# The debug build: the same sources with MUON_DEBUG, whose streaming kernels
# check every tile against the extents of the tables (error code 16 instead
# of an out-of-bounds access).  Built only on request.
BUILD_DEBUG = os.path.join(HERE, "_build_debug")
LIB_DEBUG = os.path.join(HERE, "libmuon_debug.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libmuon")
    return path


def _build_binding() -> None:
    """The C half of the Python binding, against this Python (its suffix keeps
    another one from loading it)."""
    src = os.path.join(CSRC, "binding.c")
    out = os.path.join(HERE, "_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
    deps = [src, os.path.join(ROOT, "include", "muon.h"), __file__]
    if os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in deps):
        return
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        warnings.warn(f"no Python.h in {include}: the embedding and loss calls are not built for Python",
                      RuntimeWarning)
        return
    cmd = [shutil.which("gcc") or "cc", "-O2", "-std=c11", "-shared", "-fPIC", "-I", include, src,
           "-o", out + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling the Python binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(out + ".tmp", out)


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib=LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [__file__]
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, extra, build_dir=BUILD) -> str:
    obj = os.path.join(build_dir, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip() and os.environ.get("MUON_BUILD_VERBOSE"):
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose: bool = False, extra=(), debug: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link libmuon.so (with
    debug: libmuon_debug.so, built with MUON_DEBUG)."""
    lib, build_dir = (LIB_DEBUG, BUILD_DEBUG) if debug else (LIB, BUILD)
    if force or _stale(lib):
        _build_library(lib, build_dir, verbose, extra, debug)
    _build_binding()
    return lib


def _build_library(lib, build_dir, verbose, extra, debug) -> None:
    os.makedirs(build_dir, exist_ok=True)
    extra = list(extra) + (["-DMUON_DEBUG"] if debug else [])
    if verbose:
        extra += ["-Xptxas", "-v"]
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra, build_dir), sources()))
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
