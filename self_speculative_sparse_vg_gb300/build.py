"""Build libvg.so (the C-ABI library) in-tree with nvcc for sm_103a, and
vg_binding.so, the native part of its Python binding.

Each .cu file is compiled to an object in parallel, then linked into
self_speculative_sparse_vg_gb300/libvg.so, which knows nothing of torch or
Python.  vg_binding.so reads tensors through torch's headers and links to
libvg.so beside it; where its headers or libraries are not installed it is left
out, with a warning: the calls that fill the cache then raise, the others work.
No cmake.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libvg.so")
BINDING = os.path.join(PKG, "vg_binding.so")
CXX = os.environ.get("CXX", "g++")
SOURCES = ["vg_host.cu", "verify.cu", "select.cu", "sparse_draft.cu", "step_tables.cu",
           "rope_append.cu", "chunk.cu", "cross.cu", "beam_select.cu", "beam_tables.cu", "copy_pages.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _torch_dir() -> str:
    return list(importlib.util.find_spec("torch").submodule_search_locations)[0]


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def binding_lacks() -> str:
    """What vg_binding.so would need that is not installed here; "" for nothing."""
    if not shutil.which(CXX):
        return f"a C++ compiler ({CXX})"
    if importlib.util.find_spec("torch") is None:
        return "torch"
    for path in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                 os.path.join(_torch_dir(), "include", "c10", "cuda", "CUDAGuard.h"),
                 os.path.join(_torch_dir(), "lib", "libc10_cuda.so")):
        if not os.path.exists(path):
            return path
    return ""


def _compile_binding() -> str:
    obj, inc = os.path.join(BUILD, "vg_binding.o"), os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    _run([CXX, "-O2", "-std=c++17", "-fPIC", "-I", sysconfig.get_paths()["include"], "-isystem", inc,
          "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-c",
          os.path.join(CSRC, "vg_binding.cpp"), "-o", obj], "vg_binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    lib = os.path.join(_torch_dir(), "lib")
    _run([CXX, "-shared", "-o", BINDING + ".tmp", obj, "-L", PKG, "-l:libvg.so", "-L", lib, "-lc10",
          "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN:" + lib],
         "link of vg_binding.so")
    os.replace(BINDING + ".tmp", BINDING)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    lacks = binding_lacks()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = None if lacks else ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    _run([nvcc(), *ARCH, "-shared", "-o", LIB + ".tmp", *objs], "link")
    os.replace(LIB + ".tmp", LIB)
    if lacks:
        if os.path.exists(BINDING):   # one of another libvg.so
            os.remove(BINDING)
        warnings.warn(f"vg_binding.so is left out: {lacks} is missing; the calls that fill the cache need it")
    else:
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
