"""Compile libmuon.so (the CUDA kernels and the C ABI) in-tree for sm_103a.

Each translation unit is compiled by its own nvcc process in parallel, then
linked into ``_lib/libmuon.so`` next to this file with the CUDA runtime linked
statically.  ``build(checked=True)`` makes ``_lib/libmuon_checked.so`` from the
same sources with ``-DMUON_DEVICE_CHECKS``: the kernels then test, before each
access that would fault if it broke, the invariants they rely on, and report a
broken one as MUON_ERR_DEVICE instead of making the access.  ``_lib/muon_ops.so``
is the binding of the operators around the step (csrc/binding.cpp, against the
installed torch; not made where there is none, since the library does not need
it).  A rebuild is skipped when the library is newer than every source and
header, and for the binding when it was made for the torch and Python that are
installed.
"""

from __future__ import annotations

import concurrent.futures
import importlib.metadata
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
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libmuon.so")
LIB_CHECKED = os.path.join(OUT_DIR, "libmuon_checked.so")
BINDING = os.path.join(OUT_DIR, "muon_ops.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
SOURCES = ["api.cu", "elementwise.cu", "gemm_tc.cu", "gemm_f32.cu", "ns_static.cu", "host_stream.cu",
           "ffn.cu", "ffn_tc.cu", "ffn_few.cu", "norm.cu", "logprobs.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date(checked: bool = False) -> bool:
    lib = LIB_CHECKED if checked else LIB
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build_binding(force: bool = False) -> str | None:
    """Build muon_ops.so if needed and return its path; None without PyTorch, whose tensors it binds."""
    if importlib.util.find_spec("torch") is None:
        return None
    inputs = [BINDING_SOURCE, os.path.join(INCLUDE, "muon.h"), os.path.abspath(__file__)]
    # what its ABI depends on besides, kept beside it
    stamp, built_for = BINDING + ".for", "torch %s, python %d.%d" % (importlib.metadata.version("torch"),
                                                                     *sys.version_info[:2])
    if not force and os.path.exists(BINDING) and os.path.exists(stamp) and open(stamp).read() == built_for and \
            all(os.path.getmtime(f) <= os.path.getmtime(BINDING) for f in inputs):
        return BINDING
    import torch
    home = os.path.dirname(torch.__file__)
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = f"{BINDING}.{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-I", INCLUDE, "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"), BINDING_SOURCE, "-o", tmp,
           "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(built_for)
    return BINDING


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """Build libmuon.so (or, checked, libmuon_checked.so) and the binding if needed; returns the library's path."""
    lib = _library(force, verbose, checked)
    build_binding(force)
    return lib


def _library(force: bool, verbose: bool, checked: bool) -> str:
    lib = LIB_CHECKED if checked else LIB
    if not force and up_to_date(checked):
        return lib
    nvcc = _nvcc()
    obj_dir = os.path.join(OUT_DIR, "obj_checked" if checked else "obj")
    os.makedirs(obj_dir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose else []
    if checked:
        extra.append("-DMUON_DEVICE_CHECKS")

    def compile_one(src):
        obj = os.path.join(obj_dir, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = lib + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def build_all(force: bool = False) -> list[str]:
    """Both libraries, their translation units compiled side by side, and the binding."""
    with concurrent.futures.ThreadPoolExecutor(max_workers=3) as ex:
        libs = [ex.submit(_library, force, False, checked) for checked in (False, True)]
        binding = ex.submit(build_binding, force)
        made = [f.result() for f in libs]
        binding.result()   # its errors, once both libraries are there
    return made


if __name__ == "__main__":
    if "--all" in sys.argv:
        print(build_all(force="--force" in sys.argv))
    else:
        print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, checked="--checked" in sys.argv))
