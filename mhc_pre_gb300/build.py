"""Compiles libmhc_gb300.so in-tree with nvcc for sm_103a.

Each translation unit compiles in parallel into an object file, then nvcc
links the shared library against the shared CUDA runtime (the same
libcudart.so that PyTorch loads).  No CMake, no setuptools.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmhc_gb300.so")
CALLS = os.path.join(HERE, "_attn_calls.so")     # CPython module that calls it (given the addresses)
CALLS_FOR = os.path.join(BUILD, "py_attn.for")       # the torch and Python that it was compiled for

SOURCES = ["mhc_abi.cu", "kernels_fwd.cu", "kernels_bwd.cu", "pre_tc.cu", "pre_bwd_tc.cu",
           "pre_bwd_fused.cu",
           "pre_bwd_noalloc.cu", "post_pre_tc.cu",
           "post_norm.cu", "pre_small.cu",
           "qk_norm_rope.cu", "qk_norm_rope_bwd.cu", "paged_attn.cu",
           "paged_attn_tc.cu", "attn_abi.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
         "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand) and shutil.which(cand) is None:
        raise RuntimeError("nvcc not found: the mHC library needs the CUDA toolkit to build")
    return cand


def _cuda_lib_dir(nvcc: str) -> str:
    root = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    for sub in ("lib64", "lib", os.path.join("targets", "sbsa-linux", "lib"),
                os.path.join("targets", "x86_64-linux", "lib")):
        d = os.path.join(root, sub)
        if os.path.exists(os.path.join(d, "libcudart.so")):
            return d
    return os.path.join(root, "lib64")


def _compile(nvcc: str, src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc, *ARCH, *FLAGS, *extra, "-I", INCLUDE, "-c",
           os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _gxx(cmd, what: str) -> None:
    r = subprocess.run(["g++", *cmd], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {what}:\n{r.stdout}\n{r.stderr}")


def calls_made_for() -> str:
    """What the Python module is compiled against: it uses torch's C++ classes,
    which no other torch or Python can be trusted to share."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def _calls_missing() -> str | None:
    """What this machine lacks to compile the Python module, if anything.  The
    library needs none of it."""
    try:
        import torch
    except ImportError:
        return "torch"
    root = os.path.dirname(torch.__file__)
    for path in (os.path.join(root, "include", "torch", "csrc", "autograd", "python_variable.h"),
                 os.path.join(root, "lib", "libc10_cuda.so"),
                 os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(path):
            return path
    return None if shutil.which("g++") else "g++"


def _build_calls(nvcc: str, made_for: str) -> None:
    """The Python module of the attention sublayer's calls."""
    import torch
    root = os.path.dirname(torch.__file__)
    headers = os.path.join(root, "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    src, obj, tmp = os.path.join(CSRC, "py_attn.cpp"), os.path.join(BUILD, "py_attn.o"), CALLS + ".tmp"
    _gxx(["-std=c++17", "-O2", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          f'-DMHC_CALLS_MADE_FOR="{made_for}"', "-I", sysconfig.get_paths()["include"],
          "-I", os.path.join(cuda, "include"), "-isystem", headers,
          "-isystem", os.path.join(headers, "torch", "csrc", "api", "include"),
          "-c", src, "-o", obj], src)
    _gxx(["-shared", "-o", tmp, obj, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
          "-lc10"], "the Python module's link")
    os.replace(tmp, CALLS)
    with open(CALLS_FOR, "w") as f:
        f.write(made_for)


def _fresh(target: str, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def _calls_fresh(made_for: str, deps) -> bool:
    if not _fresh(CALLS, deps) or not os.path.exists(CALLS_FOR):
        return False
    with open(CALLS_FOR) as f:
        return f.read() == made_for


def _build_library(nvcc: str, extra) -> None:
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(nvcc, s, extra), SOURCES))
    libdir = _cuda_lib_dir(nvcc)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-L", libdir, "-Xlinker", "-rpath", "-Xlinker", libdir]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(verbose: bool = False, extra_flags=()) -> str:
    """Builds the library and its Python module where a source is newer than
    they are, and the module also for another torch or Python; returns the
    library's path.  Without torch's headers, Python's or g++ the library is
    built alone, and the binding says that its module is missing."""
    os.makedirs(BUILD, exist_ok=True)
    module = os.path.join(CSRC, "py_attn.cpp")
    shared = [os.path.join(INCLUDE, "mhc.h"), os.path.abspath(__file__)]
    sources = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    sources.remove(module)
    missing = _calls_missing()
    lib_due = bool(extra_flags) or not _fresh(LIB, sources + shared)
    made_for = None if missing else calls_made_for()
    calls_due = made_for is not None and not _calls_fresh(made_for, [module, *shared])
    if lib_due or calls_due:
        nvcc = _nvcc()
        with cf.ThreadPoolExecutor(max_workers=2) as ex:
            jobs = [ex.submit(_build_library, nvcc, list(extra_flags))] if lib_due else []
            jobs += [ex.submit(_build_calls, nvcc, made_for)] if calls_due else []
        for job in jobs:
            job.result()
        if verbose:
            print(f"built {LIB}")
    if missing:
        print(f"the attention sublayer's Python calls are not built: {missing} is missing", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
