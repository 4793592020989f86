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
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmhc_gb300.so")
CALLS = os.path.join(HERE, "_attn_calls.so")     # CPython module that calls it (given the addresses)

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


def _compile_calls(nvcc: str) -> str:
    """The object of the Python module of the attention sublayer's calls."""
    import torch
    src, obj = os.path.join(CSRC, "py_attn.cpp"), os.path.join(BUILD, "py_attn.o")
    if os.path.exists(obj) and all(os.path.getmtime(d) <= os.path.getmtime(obj)
                                   for d in (src, os.path.join(INCLUDE, "mhc.h"), os.path.abspath(__file__))):
        return obj
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    headers = os.path.join(os.path.dirname(torch.__file__), "include")
    _gxx(["-std=c++17", "-O2", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), "-isystem", headers,
          "-isystem", os.path.join(headers, "torch", "csrc", "api", "include"), "-c", src, "-o", obj], src)
    return obj


def _link_calls(obj: str) -> None:
    import torch
    tmp = CALLS + ".tmp"
    _gxx(["-shared", "-o", tmp, obj, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], "the Python module's link")
    os.replace(tmp, CALLS)


def build(verbose: bool = False, extra_flags=()) -> str:
    """Builds the library and its Python module if any source is newer than
    they are; returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(INCLUDE, "mhc.h"))
    deps.append(os.path.abspath(__file__))
    if os.path.exists(LIB) and os.path.exists(CALLS) and not extra_flags:
        lib_mtime = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
        if all(os.path.getmtime(d) <= lib_mtime for d in deps):
            return LIB
    nvcc = _nvcc()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_compile_calls, nvcc)
        objs = list(ex.map(lambda s: _compile(nvcc, s, list(extra_flags)), SOURCES))
    libdir = _cuda_lib_dir(nvcc)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-L", libdir, "-Xlinker", "-rpath", "-Xlinker", libdir]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_calls(calls.result())
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
