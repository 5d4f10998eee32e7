"""Build libsage_gb300.so (sm_103a) in-tree with nvcc.

Each CUDA translation unit is compiled in parallel, then linked into one
shared library next to this file.  Beside it the host compiler makes
_sage_binding-torch<version><suffix>.so, the CPython module that hands torch
tensors to the page-cache entries; without torch there is no such module, and
the C library is built alone.  No cmake, no torch extension machinery.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsage_gb300.so")
SOURCES = ["sage_api.cu", "sage_prep.cu", "sage_attn.cu", "sage_noalloc.cu", "sage_tables.cu", "sage_paged.cu",
           "sage_paged_tiles.cu", "sage_paged_tiles_tree.cu", "sage_paged_tiles_half.cu", "sage_rotary.cu", "sage_tree.cu"]
BINDING_SOURCE = os.path.join(CSRC, "sage_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def binding_path() -> str | None:
    """The tensor-marshalling module of the torch and Python that run this (None
    without torch, which users of the C library may lack).  It reads tensors by
    the layout of one torch and links against one Python, so its name holds both
    versions (and, in Python's suffix, the machine): after a change of either,
    what was built before is not loaded."""
    try:
        import torch
    except ImportError:
        return None
    return os.path.join(PKG, f"_sage_binding-torch{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _compile_binding() -> None:
    """The tensor-marshalling module, against the torch and Python that run this."""
    import torch
    root = os.path.dirname(torch.__file__)
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler found")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    out = binding_path()
    tmp = out + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(root, "include"), "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", cuda, "-I", INCLUDE, BINDING_SOURCE, "-o", tmp, "-L", os.path.join(root, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for sage_binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _stale() -> bool:
    made = [m for m in (LIB, binding_path()) if m is not None]
    if not all(os.path.exists(m) for m in made):
        return True
    t = min(os.path.getmtime(m) for m in made)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding) if binding_path() is not None else None
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if binding is not None:
        binding.result()                                   # raises what failed; the C library stands by itself
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
