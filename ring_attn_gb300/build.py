"""Builds libringattn.so in-tree for sm_103a (nvcc, one translation unit per kernel family, in parallel),
and _ra_binding.so (the host compiler), which marshals torch tensors into its cache calls.  The
library needs nvcc alone; where torch is not installed, only it is built.

build(debug_bounds=True) builds the debug variant libringattn_dbg.so instead:
the same sources compiled with RA_DEBUG_BOUNDS, under which every kernel checks
its tiled-copy coordinates and global row indices against the tensor extents
and reports a violation as RA_ERR_DEVICE (with the site) instead of making the
access.  The binding loads it when RA_LIB_VARIANT=debug_bounds is set."""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libringattn.so")
BUILD_DBG = os.path.join(PKG, "_build_dbg")
LIB_DBG = os.path.join(PKG, "libringattn_dbg.so")
SOURCES = ["ra_api.cu", "ra_fwd.cu", "ra_bwd.cu", "ra_dkdv_pair.cu", "ra_simple.cu", "ra_cache.cu", "ra_cache_attn.cu",
           "ra_cache_chunk.cu"]
HEADERS = [os.path.join(CSRC, h) for h in ("ra_device.cuh", "ra_internal.h", "ra_tiles.cuh", "ra_bwd_common.cuh",
                                               "ra_cache_args.h", "ra_cache.cuh", "ra_cache_line.cuh")] + [
    os.path.join(ROOT, "include", "ringattn.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]


BINDING_SRC = os.path.join(CSRC, "ra_binding.cpp")
BINDING = os.path.join(PKG, "_ra_binding.so")
BINDING_NOTE = os.path.join(BUILD, "binding.txt")


def _binding_cmd():
    """The compiler's command line, or None where there is no torch to build against."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    t = os.path.dirname(os.path.abspath(spec.origin))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-w", "-o", BINDING, BINDING_SRC,
            *("-I" + i for i in inc if os.path.isdir(i)), "-L" + os.path.join(t, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]


def _binding_made_for(cmd) -> str:
    """What _ra_binding.so depends on besides its sources: the command, and torch's version and Python's."""
    with open(os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "version.py")) as f:
        return "\n".join([*cmd, f.read(), sys.version])


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libringattn.so")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("build step failed:\n" + " ".join(cmd) + "\n" + r.stdout)
    return r.stdout


def build(verbose: bool = False, force: bool = False, debug_bounds: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link libringattn.so (or, with
    debug_bounds, libringattn_dbg.so); returns its path."""
    nvcc = _nvcc()
    bdir, lib = (BUILD_DBG, LIB_DBG) if debug_bounds else (BUILD, LIB)
    extra = ["-DRA_DEBUG_BOUNDS"] if debug_bounds else []
    os.makedirs(bdir, exist_ok=True)
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(bdir, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + HEADERS):
            cmd = [nvcc] + ARCH + FLAGS + extra + (["-Xptxas", "-v"] if verbose else []) + ["-c", s, "-o", o]
            jobs.append(cmd)
    binding = _binding_cmd()
    made_for = _binding_made_for(binding) if binding else ""
    if not (binding and (force or _read(BINDING_NOTE) != made_for
                         or _stale(BINDING, [BINDING_SRC, os.path.join(ROOT, "include", "ringattn.h")]))):
        binding = None
    with ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        marshaller = ex.submit(_run, binding) if binding else None
        for out in ex.map(_run, jobs):
            if verbose and out:
                sys.stdout.write(out)
    if force or jobs or _stale(lib, objs):
        _run([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", lib] + objs)
    if marshaller:
        marshaller.result()  # raises what went wrong; the library is there all the same
        os.makedirs(os.path.dirname(BINDING_NOTE), exist_ok=True)
        with open(BINDING_NOTE, "w") as f:
            f.write(made_for)
    return lib


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv, debug_bounds="--debug-bounds" in sys.argv))
