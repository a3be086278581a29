"""Build the CUDA library ``libdiffattn.so`` in-tree for sm_100a.

Each ``csrc/*.cu`` is compiled by nvcc into ``_build/`` (in parallel), then
linked into ``differential_attention_04_b200/libdiffattn.so``.  Run as
``python -m differential_attention_04_b200.build``; ``--verbose-ptxas`` prints
register / shared-memory usage per kernel.  ``--debug`` builds the
bounds-checked variant instead (``-DDIFFATTN_DEBUG``, objects in
``_build_debug/``, library ``libdiffattn_debug.so``): its kernels check every
global index and tensor-map coordinate, skip an access out of range and
record DIFFATTN_ERR_BOUNDS in the status word.  ``csrc/marshal.cpp`` becomes the
Python module ``_marshal`` (g++, against torch's headers), which marshals the
calls that a server makes every step; where torch or a header is missing the
library is built all the same.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdiffattn.so")
BUILD_DEBUG = os.path.join(ROOT, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libdiffattn_debug.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _needs_build(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    deps = [src] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def build_marshal(force: bool = False) -> str | None:
    """The marshalling module, in-tree; its torch symbols are those of the torch that imports it.

    None where it cannot be built (the library needs neither torch nor Python): the binding then marshals every
    call itself, and a module of older sources is taken away."""
    src, header = os.path.join(CSRC, "marshal.cpp"), os.path.join(INCLUDE, "diffattn.h")
    spec = importlib.util.find_spec("torch")
    torch_dir = os.path.dirname(spec.origin) if spec and spec.origin else None
    needed = [src, header] + ([os.path.join(torch_dir, "version.py")] if torch_dir else [])
    if not force and os.path.exists(MARSHAL) and \
            all(os.path.exists(f) and os.path.getmtime(f) <= os.path.getmtime(MARSHAL) for f in needed):
        return MARSHAL
    python_h, cxx = sysconfig.get_paths()["include"], shutil.which("g++")
    missing = [what for what, there in (
        ("torch with CUDA", torch_dir and os.path.exists(os.path.join(torch_dir, "lib", "libc10_cuda.so"))),
        ("torch's headers", torch_dir and os.path.isdir(os.path.join(torch_dir, "include"))),
        ("Python's headers", os.path.exists(os.path.join(python_h, "Python.h"))), ("g++", cxx)) if not there]
    if not missing:
        cuda = os.path.dirname(os.path.dirname(_nvcc()))
        tmp = MARSHAL + ".tmp"
        cmd = [cxx, "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", src, "-o", tmp, "-I", INCLUDE,
               "-isystem", os.path.join(torch_dir, "include"), "-isystem", os.path.join(cuda, "include"),
               "-isystem", python_h, "-L", os.path.join(torch_dir, "lib"),
               "-lc10", "-ltorch_cpu", "-ltorch_python", "-lc10_cuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode == 0:
            os.replace(tmp, MARSHAL)
            return MARSHAL
        sys.stderr.write(r.stdout + r.stderr)
        missing = [f"g++ failed on {src}"]
    sys.stderr.write(f"the marshalling module was not built ({', '.join(missing)}); the binding does without\n")
    if os.path.exists(MARSHAL):
        os.remove(MARSHAL)
    return None


def build(verbose_ptxas: bool = False, force: bool = False, debug: bool = False) -> str:
    nvcc = _nvcc()
    bdir, lib = (BUILD_DEBUG, LIB_DEBUG) if debug else (BUILD, LIB)
    os.makedirs(bdir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                    "--expt-relaxed-constexpr"]
    if debug:
        flags += ["-DDIFFATTN_DEBUG"]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(bdir, os.path.basename(src).replace(".cu", ".o"))
        if force or verbose_ptxas or _needs_build(obj, src):
            cmd = [nvcc, "-c", src, "-o", obj] + flags
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0 or verbose_ptxas:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    if force or not os.path.exists(lib) or any(os.path.getmtime(o) > os.path.getmtime(lib) for o in objs):
        tmp = lib + ".tmp"
        cmd = [nvcc, "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, lib)
    if not debug:
        build_marshal(force)
    return lib


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--debug", action="store_true", help="the bounds-checked library")
    a = ap.parse_args()
    print(build(a.verbose_ptxas, a.force, a.debug))
