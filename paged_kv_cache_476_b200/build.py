"""Build libpagedkv.so in-tree with nvcc for sm_100a.

Usage: ``python paged_kv_cache_476_b200/build.py [--force]`` (run it as a
file: importing the package first would load a possibly stale library).  Each ``.cu``
under ``csrc/`` compiles with nvcc and each host-only ``.cpp`` with g++ to an
object in ``_build/`` (in parallel), then the
objects link into ``paged_kv_cache_476_b200/libpagedkv.so`` with the CUDA
runtime linked statically.  nvcc cross-compiles, so no GPU is needed.
``csrc/python/binding.cpp`` becomes the CPython module ``_binding`` next to it
(g++ against torch's headers; the library itself knows nothing of torch).
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.metadata
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")
BINDING_SRC = os.path.join(CSRC, "python", "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-Xptxas", "-O3",
         f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]


CXX = os.environ.get("CXX", "g++")
CXXFLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", f"-I{os.path.join(ROOT, 'include')}"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _read(path):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def check_registers(source: str, log: str) -> None:
    """Kernels that exchange registers (setmaxnreg) count on what their block is launched
    with, ``kLaunchRegs`` in the source, of a compiler that is free to allot fewer: an
    exchange that asks for more than the block has would wait for ever.  The launch
    refuses such a kernel; this says so where it can be acted on.  ``log`` is what
    ptxas -v prints."""
    want = re.search(r"\bkLaunchRegs = (\d+)", source)
    if not want:
        return
    kernels = re.findall(r"Compiling entry function '(\S*prefix_kernel\S*)'.*?Used (\d+) registers",
                         log, re.S)
    quantised = [(k, int(n)) for k, n in kernels if not re.search(r"prefix_kernelILi\d+ELi0E", k)]
    if not quantised:
        raise RuntimeError("no registers of the quantised prefix kernels in the compiler's output")
    for kernel, n in quantised:
        if n < int(want[1]):
            raise RuntimeError(f"{kernel} was compiled to {n} registers, its register exchange "
                               f"counts on {want[1]} (kLaunchRegs, with the split beside it)")


def _compile(src, extra):
    obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
    if _stale(obj, [src, *_headers()]) or extra.get("force"):
        if src.endswith(".cpp"):  # host-only runtime code
            cmd = [CXX, *CXXFLAGS, "-c", src, "-o", obj]
        else:
            cmd = [NVCC, *ARCH, *FLAGS, *extra.get("flags", []), "-c", src, "-o", obj]
            source = _read(src)
            if "kLaunchRegs" in source and "-v" not in cmd:
                cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if src.endswith(".cu"):
            try:
                check_registers(source, r.stdout + r.stderr)
            except RuntimeError:
                os.unlink(obj)
                raise
        return obj, r.stderr
    return obj, ""


def binding_key() -> str:
    """What the CPython module is built against: it reads tensors through torch's inline
    code, so it goes with one torch and one Python."""
    return (f"torch {importlib.metadata.version('torch')}, "
            f"{sysconfig.get_config_var('SOABI') or sys.version}")


def _build_binding(force):
    """The CPython module; torch is located without importing it.  It carries its key and
    is built again where that or the command changes (kept beside the objects)."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    tmp = BINDING + f".tmp{os.getpid()}"
    dirs = [os.path.join(ROOT, "include"), os.path.join(torch, "include"),
            os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
            sysconfig.get_paths()["include"]]
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared", *(f"-I{d}" for d in dirs),
           f'-DPKV_BINDING_KEY="{binding_key()}"', BINDING_SRC, "-L" + os.path.join(torch, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    made_by = os.path.join(BUILD, "binding.cmd")
    want = "\n".join(cmd)
    if not force and not _stale(BINDING, [BINDING_SRC, *_headers()]) and _read(made_by) == want:
        return
    r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(made_by, "w") as f:
        f.write(want)


def build(force: bool = False, verbose: bool = False, flags=()) -> str:
    """Compile every CUDA source and link ``libpagedkv.so``; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    extra = {"force": force, "flags": list(flags)}
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        binding = ex.submit(_build_binding, force)
        results = list(ex.map(lambda s: _compile(s, extra), srcs))
        binding.result()
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            if log:
                print(log, file=sys.stderr)
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    verbose = "-v" in sys.argv
    fl = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force=force, verbose=verbose or bool(fl), flags=fl))
