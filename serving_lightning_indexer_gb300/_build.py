"""In-tree build of libcsa2.so for sm_103a with nvcc, and of the Python extension
_csa2_call.so over it with g++ and torch's headers (no cmake).

Each translation unit compiles in parallel; the objects are linked into
``serving_lightning_indexer_gb300/_lib/``.  A rebuild happens only when a source
or header is newer than its library, or torch or Python are not those that the
extension was built with.  The library alone needs neither of them, nor g++.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "_lib")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(LIBDIR, "libcsa2.so")
CALL = os.path.join(LIBDIR, "_csa2_call.so")   # Python extension: binding.cpp
CALL_MADE_WITH = os.path.join(LIBDIR, "_csa2_call.made_with")
SOURCES = ["csa2_api.cu", "index_score.cu", "select.cu", "sparse_attn.cu", "compress.cu", "topk_noalloc.cu",
           "quant_fp8.cu", "fp8_linear.cu", "batch_plan.cu", "add_norm.cu", "lora.cu", "logprobs.cu"]
HEADERS = [os.path.join(ROOT, "include", "csa2.h")] + [
    os.path.join(CSRC, f) for f in ("csa2_device.cuh", "csa2_rope.cuh", "csa2_e4m3.cuh", "csa2_internal.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def _cuda_home() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))


def made_with() -> str:
    """What the extension's binary interface is of: this Python and this torch."""
    import torch
    return f"{sys.implementation.cache_tag}, torch {torch.__version__}"


def call_made_with() -> str | None:
    """The same of the built extension, None if there is none or it does not say."""
    if not os.path.exists(CALL) or not os.path.exists(CALL_MADE_WITH):
        return None
    with open(CALL_MADE_WITH) as f:
        return f.read()


def _compile_call(verbose: bool) -> str:
    """Compile binding.cpp; returns its object."""
    import torch
    src, obj = os.path.join(CSRC, "binding.cpp"), os.path.join(OBJDIR, "binding.o")
    include = os.path.join(os.path.dirname(torch.__file__), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *(f"-I{d}" for d in (include, os.path.join(include, "torch", "csrc", "api", "include"),
                               os.path.join(_cuda_home(), "include"), sysconfig.get_paths()["include"])),
          "-c", src, "-o", obj], src, verbose)
    return obj


def _link_call(obj: str, verbose: bool) -> None:
    import torch
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run(["g++", "-shared", "-o", CALL + ".tmp", obj, f"-L{LIBDIR}", "-lcsa2", "-Wl,-rpath,$ORIGIN", f"-L{torch_lib}",
          "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{torch_lib}",
          f"-L{os.path.join(_cuda_home(), 'lib64')}", "-lcudart"], "_csa2_call.so", verbose)
    if os.path.exists(CALL_MADE_WITH):
        os.remove(CALL_MADE_WITH)  # says nothing of what is about to be there
    os.replace(CALL + ".tmp", CALL)
    with open(CALL_MADE_WITH, "w") as f:
        f.write(made_with())


def _run(cmd: list[str], what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {what}:\n{r.stdout}\n{r.stderr}")


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CSA2 library needs the CUDA toolkit to build")


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA sources and link libcsa2.so; returns its path."""
    os.makedirs(LIBDIR, exist_ok=True)
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    if not force and not _stale(LIB, srcs + HEADERS):
        return LIB
    cc = nvcc()

    def one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src).replace(".cu", ".o"))
        if force or _stale(obj, [src] + HEADERS):
            _run([cc, *ARCH, *FLAGS, "-c", src, "-o", obj], src, verbose)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(one, srcs))
    _run([cc, *ARCH, "-shared", "-o", LIB + ".tmp", *objs], "libcsa2.so", verbose)
    os.replace(LIB + ".tmp", LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """Build libcsa2.so and _csa2_call.so; returns the former's path."""
    call_stale = force or _stale(CALL, [os.path.join(CSRC, "binding.cpp"), HEADERS[0]]) or call_made_with() != made_with()
    if not call_stale:
        return build_library(force, verbose)
    os.makedirs(OBJDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:   # beside the library
        obj = ex.submit(_compile_call, verbose)
        build_library(force, verbose)
        _link_call(obj.result(), verbose)
    return LIB


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
    try:
        import torch  # noqa: F401
    except ImportError:
        print("no torch: _csa2_call.so is not built")
    else:
        build(verbose=True)
