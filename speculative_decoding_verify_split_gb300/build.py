"""Builds the C-ABI library ``_lib/libverify_attn.so`` in-tree with nvcc, and the
Python extension ``_lib/va_binding.so`` over it with the host compiler.

Every translation unit is compiled for sm_103a only, in parallel, then linked
into one shared object with the CUDA runtime linked statically (so the
library loads on a machine without a GPU driver; only the kernels need one).
Run ``python -m speculative_decoding_verify_split_gb300.build`` or call
``build_library()``.
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
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libverify_attn.so")
BINDING = os.path.join(LIBDIR, "va_binding.so")
BINDING_SOURCE = "va_binding.cpp"
BINDING_STAMP = os.path.join(LIBDIR, "va_binding.abi")  # the torch and Python that BINDING was built for

SOURCES = ["va_host.cpp", "va_host_append.cpp", "va_host_chunk.cpp", "va_host_pages.cpp", "va_main_tc.cu", "va_mla_tc.cu", "va_mla_bf16_tc.cu", "va_merge.cu",
           "va_noalloc.cu", "va_pagetable.cu", "va_append.cu", "va_chunk.cu",
           "va_pages.cu"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler",
          "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build the library")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *COMMON, "-Xptxas", "-v" if verbose else "-O3", "-c",
           os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd.insert(1, "-x")
        cmd.insert(2, "cu")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def _compile_binding(verbose: bool) -> str:
    """The extension's object: the torch headers of the running interpreter."""
    import torch

    tdir = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, BINDING_SOURCE + ".o")
    cxx = shutil.which("g++") or "g++"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(tdir, "include"), "-isystem",
           os.path.join(tdir, "include", "torch", "csrc", "api", "include"), "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"],
           "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SOURCE}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def _link_binding(obj: str) -> None:
    """Links the extension against the library beside it and the torch libraries
    that the interpreter has loaded."""
    import torch

    tlib = os.path.join(os.path.dirname(os.path.abspath(torch.__file__)), "lib")
    tmp = BINDING + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", obj, "-o", tmp, "-L", LIBDIR, "-lverify_attn", "-L", tlib, "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING)


def binding_abi() -> str:
    """What the extension is built against: another torch or interpreter reads its
    tensors with another layout."""
    import torch

    return f"torch {torch.__version__} cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} python {sysconfig.get_config_var('SOABI')}"


def _older(target: str, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps if os.path.exists(d))


_COMMON_DEPS = [os.path.join(ROOT, "include", "verify_attn.h"), os.path.abspath(__file__)]


def library_stale() -> bool:
    return _older(LIB, _COMMON_DEPS + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != BINDING_SOURCE])


def binding_stale() -> bool:
    if _older(BINDING, _COMMON_DEPS + [os.path.join(CSRC, BINDING_SOURCE)]) or not os.path.exists(BINDING_STAMP):
        return True
    try:
        with open(BINDING_STAMP) as f:
            return f.read() != binding_abi()
    except ImportError:  # no torch here: building the extension says so, behind the library
        return True


def build_library(force: bool = False, verbose: bool = False) -> str:
    lib, binding = force or library_stale(), force or binding_stale()
    if not lib and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding_obj = ex.submit(_compile_binding, verbose) if binding else None
        if lib:
            objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
            tmp = LIB + ".tmp"
            cmd = [nvcc(), *ARCH, "-shared", "-Xlinker", "--exclude-libs,ALL", *objs, "-o", tmp]
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
            os.replace(tmp, LIB)  # whether or not the extension compiles
        if binding:
            _link_binding(binding_obj.result())
            with open(BINDING_STAMP, "w") as f:
                f.write(binding_abi())
    return LIB


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
