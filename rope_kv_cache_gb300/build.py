"""Build libropekv.so (the C ABI and its sm_103a kernels) in-tree with nvcc,
libropekv_serving.so (the serving operators around the paged cache) with
ropekv_bind-*.so, its Python module for torch tensors, and libropekv_floor.so, the
copy kernel the benchmark times as the floor of a decode-sized launch.

Each library is compiled for sm_103a only and linked against the static CUDA
runtime, so it loads without any other file from this package (the Python module
needs libropekv_serving.so beside it); all translation units compile in parallel.
Output: ``rope_kv_cache_gb300/lib/`` (git-ignored).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libropekv.so")
FLOOR_LIB_PATH = os.path.join(LIB_DIR, "libropekv_floor.so")
SERVING_LIB_PATH = os.path.join(LIB_DIR, "libropekv_serving.so")
SOURCES = [os.path.join(CSRC, "ropekv_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, "ropekv_kernels.cuh"), os.path.join(INCLUDE, "ropekv.h")]
FLOOR_SOURCES = [os.path.join(CSRC, "ropekv_floor.cu")]
FLOOR_DEPS = FLOOR_SOURCES + [os.path.join(INCLUDE, "ropekv_floor.h")]
SERVING_SOURCES = [os.path.join(CSRC, "ropekv_serving.cu"),
                   os.path.join(CSRC, "ropekv_attention.cu")]
SERVING_DEPS = SERVING_SOURCES + [os.path.join(CSRC, n) for n in (
    "ropekv_kernels.cuh", "ropekv_attention_kernels.cuh", "ropekv_prefix_kernel.cuh")] + [
    os.path.join(INCLUDE, n) for n in ("ropekv.h", "ropekv_serving.h")]
BIND_SOURCE = os.path.join(CSRC, "ropekv_bind.cpp")
BIND_DEPS = [BIND_SOURCE] + [os.path.join(INCLUDE, n) for n in ("ropekv.h", "ropekv_serving.h")]
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libropekv.so")


def nvcc_command(out: str, extra=(), sources=None) -> list:
    return [nvcc(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared",
            "-Xcompiler", "-fPIC,-fvisibility=hidden", "-cudart", "static",
            "-I", INCLUDE, "-I", CSRC, *extra, "-o", out, *(sources or SOURCES)]


def bind_path() -> str:
    """The Python module for the running torch and Python. Its name holds both: it is tied
    to torch's C++ ABI, which file times say nothing about, so that after another torch was
    installed the module is missing (and built again) instead of loaded."""
    import torch

    return os.path.join(LIB_DIR, f"ropekv_bind-torch{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def bind_lacks() -> str:
    """What the Python module needs and this machine does not have ("" if nothing)."""
    try:
        import torch
    except ImportError:
        return "torch"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    lib = os.path.join(os.path.dirname(os.path.abspath(torch.__file__)), "lib")
    return "" if os.path.exists(os.path.join(lib, "libc10_cuda.so")) else "a CUDA build of torch"


def bind_commands(out: str, obj: str) -> tuple:
    """Compile and link commands of the Python module."""
    import torch  # headers and libraries of the installed torch

    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    lib = os.path.join(root, "lib")
    compile_ = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                "-I", INCLUDE, "-isystem", os.path.join(root, "include"),
                "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                "-isystem", os.path.join(cuda, "include"),
                "-isystem", sysconfig.get_paths()["include"], "-c", "-o", obj, BIND_SOURCE]
    link = [os.environ.get("CXX", "g++"), "-shared", "-o", out, obj, "-L", LIB_DIR, "-lropekv_serving",
            "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    return compile_, link


def _stale(lib: str, deps) -> bool:
    return not os.path.exists(lib) or os.path.getmtime(lib) < max(os.path.getmtime(p) for p in deps)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Build the libraries where stale (or always with force); returns the
    path of libropekv.so. The C libraries need nvcc alone. Where the Python module's
    needs are not met it is left out with a warning, and the Python functions of the
    serving operators raise."""
    os.makedirs(LIB_DIR, exist_ok=True)
    extra = ("-Xptxas", "-v") if verbose else ()
    jobs = []   # (compilers, their objects, link command (None: nothing to link), output, library)
    for lib, sources, deps in ((LIB_PATH, SOURCES, DEPS),
                               (FLOOR_LIB_PATH, FLOOR_SOURCES, FLOOR_DEPS),
                               (SERVING_LIB_PATH, SERVING_SOURCES, SERVING_DEPS)):
        if force or _stale(lib, deps):
            tmp = lib + f".{os.getpid()}.tmp"
            if len(sources) == 1:
                jobs.append(([subprocess.Popen(nvcc_command(tmp, extra, sources))], [], None, tmp, lib))
            else:
                objs = [f"{tmp}.{i}.o" for i in range(len(sources))]
                procs = [subprocess.Popen([a for a in nvcc_command(o, (*extra, "-c"), [src])
                                           if a != "-shared"]) for o, src in zip(objs, sources)]
                jobs.append((procs, objs, nvcc_command(tmp, (), objs), tmp, lib))
    lacks = bind_lacks()
    if lacks:
        warnings.warn(f"the Python module of the serving operators is not built: {lacks} is not there")
    elif force or _stale(bind_path(), BIND_DEPS):
        bind = bind_path()
        # after the library that it links with
        tmp = bind + f".{os.getpid()}.tmp"
        compile_, link = bind_commands(tmp, tmp + ".o")
        jobs.append(([subprocess.Popen(compile_)], [tmp + ".o"], link, tmp, bind))
    failed = []
    for procs, objs, link, tmp, lib in jobs:
        ok = all([p.wait() == 0 for p in procs])
        if ok and link:
            ok = subprocess.run(link).returncode == 0
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
        if ok:
            os.replace(tmp, lib)
        else:
            failed.append(os.path.basename(lib))
    if failed:
        raise RuntimeError(f"the compiler failed for {', '.join(failed)}")
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
