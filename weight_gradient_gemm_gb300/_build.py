"""Builds libforge.so in-tree with nvcc for sm_103a (no CMake, no torch build).

Each .cu file compiles to an object in parallel, then one shared library is
linked with the CUDA runtime static.  Beside it, the Python calls of the
operators around the weight gradient (csrc/forge_call.cpp) compile to a CPython
extension against the installed torch, named for the interpreter's ABI; where
that cannot be built the library is complete without it (forge.py calls through
ctypes, a few microseconds slower).  Re-running is cheap: objects are rebuilt
only when a source or header is newer.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libforge.so")
CALL = os.path.join(PKG, "_forge_call" + sysconfig.get_config_var("EXT_SUFFIX"))
CXX = "g++"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(ROOT, "include", "forge.h"))
    return hs


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build_call() -> bool:
    """The CPython extension (host code only, the machine's own compiler); False,
    with a warning and no file, where it does not build."""
    try:
        src = os.path.join(CSRC, "forge_call.cpp")
        torch_dir = list(importlib.util.find_spec("torch").submodule_search_locations)[0]
        if not _stale(CALL, [src, os.path.join(ROOT, "include", "forge.h"),
                             os.path.join(torch_dir, "version.py")]):
            return True
        if os.path.exists(CALL):
            os.remove(CALL)
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
        inc = [os.path.join(ROOT, "include"), os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
        cmd = ([CXX, "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", src, "-o", CALL]
               + [a for i in inc for a in ("-isystem" if i is not inc[0] else "-I", i)]
               + ["-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
                  "-lc10_cuda"])
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode == 0:
            return True
        why = r.stdout + r.stderr
    except (OSError, AttributeError, RuntimeError) as e:   # no compiler, torch or headers
        why = str(e)
    warnings.warn(f"forge_call.cpp did not build, calls go through ctypes:\n{why}", stacklevel=2)
    return False


def build(verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))
    headers = _headers()
    flags = FLAGS + list(extra_flags or [])
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src[:-3] + ".o")
        path = os.path.join(CSRC, src)
        if _stale(obj, [path] + headers):
            cmd = [cc] + ARCH + flags + ["-c", path, "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
            if verbose:
                print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        call = ex.submit(build_call)
        objs = list(ex.map(compile_one, sources))
        call.result()
    if _stale(LIB, objs):
        cmd = [cc] + ARCH + ["-shared", "-cudart", "static", "-o", LIB] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose="-v" in sys.argv, extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else None))
