"""Builds libtopk_gb300.so in-tree with nvcc for sm_103a (GB300).

Each translation unit is compiled in parallel, then linked into one shared
library exporting the C ABI of include/topk.h; and, where torch is installed with
its CUDA headers and libraries, the Python module that makes language.py's calls
of it (_language_calls.so).  The library needs neither Python nor torch.  Usage:
    python -m top_selection_prof_gb300.build [--verbose]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libtopk_gb300.so")
BUILD = os.path.join(ROOT, "_build")
SOURCES = ["topk_api.cu", "kernels_sample.cu", "kernels_filter.cu", "kernels_fallback.cu", "kernels_select.cu",
           "kernels_rows.cu", "params.cpp", "topk_noalloc.cu", "ops_api.cu", "kernels_linear.cu", "kernels_mma.cu", "kernels_places.cu",
           "kernels_norm.cu", "kernels_tokens.cu", "kernels_experts.cu", "kernels_cache.cu"]
CALLS = os.path.join(HERE, "_language_calls.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the engine")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), "-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC,-O3",
           "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), res.stderr))
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def _run(cmd, what):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("%s:\n%s\n%s" % (what, " ".join(cmd), res.stderr))


def _calls_lack() -> str | None:
    """What this machine lacks for the Python module, or None."""
    import sysconfig
    try:
        import torch
    except ImportError as e:
        return "torch cannot be imported (%s)" % e
    at = os.path.dirname(torch.__file__)
    for f in (os.path.join(sysconfig.get_paths()["include"], "Python.h"), os.path.join(at, "include", "c10", "cuda", "CUDAStream.h"),
              os.path.join(at, "lib", "libc10_cuda.so"), os.path.join(at, "lib", "libtorch_cuda.so")):
        if not os.path.exists(f):
            return "there is no %s" % f
    return None


def _compile_calls() -> str:
    """The object of the Python module: host code with the headers of this machine's Python and torch."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, "language_calls.o")
    _run([shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
          "-I", sysconfig.get_paths()["include"], "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", cuda, "-c", os.path.join(CSRC, "language_calls.cpp"), "-o", obj], "g++ failed for language_calls.cpp")
    return obj


def _link_calls(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS + ".tmp"
    _run([shutil.which("g++") or "c++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:" + os.path.basename(LIB), "-L", lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10",
          "-Wl,-rpath,$ORIGIN"], "link failed for the Python module")
    os.replace(tmp, CALLS)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        lack = _calls_lack()
        calls = None if lack else ex.submit(_compile_calls)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        tmp = LIB + ".tmp"
        _run([nvcc(), "-shared", *ARCH, "-o", tmp, *objs], "link failed")
        os.replace(tmp, LIB)
        if calls:  # (the library is there, whatever becomes of the module)
            _link_calls(calls.result())
        else:
            if os.path.exists(CALLS):
                os.remove(CALLS)  # (it was linked to another library)
            sys.stderr.write("the module of language.py's calls is not built: %s\n" % lack)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
