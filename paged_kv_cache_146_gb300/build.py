"""Build libpagedkv.so in-tree with nvcc for sm_103a.

Usage: ``python -m paged_kv_cache_146_gb300.build`` (or ``__graft_entry__.build()``).
Each translation unit compiles in parallel; the shared library links the CUDA
runtime statically, so it only needs the driver at run time.  _fastcall.so beside
it holds the binding's compiled argument checks.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
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
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")
FASTCALL = os.path.join(PKG, "_fastcall.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["ledger.cpp", "cache_write.cu", "paged_decode.cu", "paged_decode_q8.cu",
           "paged_prefill.cu", "append_rope.cu", "paged_window.cu", "paged_tree.cu", "cache_compact.cu"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src: str, verbose: bool, build_dir: str = BUILD, defines=()) -> str:
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "cu"]
    cmd[1:1] = [f"-D{d}" for d in defines]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def interface_hash() -> str:
    """Of the entry points that _fastcall.so calls and of its own functions: the binding
    takes it only when it was built from the sources that are there now."""
    h = hashlib.sha256()
    for path in (os.path.join(INCLUDE, "pagedkv.h"), os.path.join(CSRC, "fastcall.cpp")):
        with open(path, "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


def _fastcall() -> None:
    """Build _fastcall.so if that can be done.  The library does not need it and the
    binding's own checks serve without it, so a failure is a warning; what an earlier
    build left is removed, as it may have been made for other signatures."""
    try:
        if _build_fastcall():
            return
    except Exception as e:                    # no compiler, headers that it cannot take
        warnings.warn(f"_fastcall.so was not built (calls of a few rows take longer): {e}")
    if os.path.exists(FASTCALL):
        os.remove(FASTCALL)


def _build_fastcall() -> bool:
    """_fastcall.so: the compiled argument checks, against torch's and Python's headers.
    False where those are not installed."""
    spec = importlib.util.find_spec("torch")
    python = sysconfig.get_paths()["include"]
    torch = spec.submodule_search_locations[0] if spec is not None else ""
    if not (os.path.exists(os.path.join(torch, "lib", "libc10_cuda.so"))
            and os.path.exists(os.path.join(python, "Python.h"))):
        return False
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = FASTCALL + ".tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-I", INCLUDE,
           f'-DPKV_INTERFACE="{interface_hash()}"',
           "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-isystem", python,
           "-isystem", os.path.join(cuda, "include"),
           os.path.join(CSRC, "fastcall.cpp"), "-o", tmp, "-L", os.path.join(torch, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on fastcall.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FASTCALL)
    return True


def build(verbose: bool = False, checked: bool = False, out: str | None = None) -> str:
    """Build the library.  ``checked=True`` compiles the kernels' bounds and
    alignment checks in (-DPKV_DEBUG_CHECKS) into ``out`` (a separate file)."""
    lib = out or LIB
    build_dir = BUILD + ("_checked" if checked else "")
    defines = ("PKV_DEBUG_CHECKS",) if checked else ()
    os.makedirs(build_dir, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        fast = None if checked or out else ex.submit(_fastcall)
        objs = list(ex.map(lambda s: _compile(s, verbose, build_dir, defines), SOURCES))
        if fast is not None:
            fast.result()
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
