"""Build libgemma_attn.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel; the shared library links the CUDA runtime
statically, so loading it needs no CUDA shared library beyond the driver. _bind.so, the native
half of the Python binding, is the one part compiled against PyTorch's headers (g++), and links
libgemma_attn.so.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgemma_attn.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BIND = os.path.join(PKG, "_bind.so")
BIND_KEY = os.path.join(BUILD, "bind.key")  # the bind_key() that _bind.so was built for
HEADER = os.path.join(ROOT, "include", "gemma_attn.h")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"] + ARCH


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgemma_attn.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer_than(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path)
                                        for d in deps + [HEADER, os.path.abspath(__file__)])


def library_up_to_date() -> bool:
    return _newer_than(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
                       glob.glob(os.path.join(CSRC, "*.h")))


def bind_key() -> str:
    """What _bind.so depends on besides its source: the interpreter and the PyTorch that it was
    compiled against and links."""
    import torch
    return "\n".join([sysconfig.get_config_var("EXT_SUFFIX") or "", sys.version, torch.__version__,
                      str(torch._C._GLIBCXX_USE_CXX11_ABI), os.path.dirname(torch.__file__)])


def bind_up_to_date() -> bool:
    if not _newer_than(BIND, [BIND_SRC]) or not os.path.exists(BIND_KEY):
        return False
    with open(BIND_KEY) as f:
        return f.read() == bind_key()


def up_to_date() -> bool:
    return library_up_to_date() and bind_up_to_date()


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _compile_bind() -> str:
    import torch
    os.makedirs(BUILD, exist_ok=True)
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "bind.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    _run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC",
          f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", os.path.dirname(HEADER), "-isystem", inc,
          "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
          "-isystem", sysconfig.get_paths()["include"], "-c", BIND_SRC, "-o", obj],
         f"g++ failed for {BIND_SRC}")
    return obj


def _link_bind(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND + f".tmp{os.getpid()}"
    _run([shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libgemma_attn.so",
          "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
          "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"], "link of _bind.so failed")
    if os.path.exists(BIND_KEY):
        os.remove(BIND_KEY)
    os.replace(tmp, BIND)
    with open(BIND_KEY, "w") as f:
        f.write(bind_key())


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """libgemma_attn.so alone: all that the calls marshalled by ctypes need."""
    if not force and library_up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([cc, "-shared", *ARCH, "-Xlinker", "-soname=libgemma_attn.so", "-o", tmp, *objs],
         "link failed")
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Both parts. If _bind.so cannot be built this raises, with the library in place."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        bind = ex.submit(_compile_bind) if force or not bind_up_to_date() else None
        build_library(force, verbose, extra_flags)
        if bind:
            _link_bind(bind.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
