"""Build the C-ABI library libmgg.so for sm_103a, in tree.

Each translation unit under csrc/ is compiled by nvcc in parallel into
_build/, then linked (static CUDA runtime, no libcuda link: the driver entry
point for tensor maps is fetched at run time) into
variable_size_expert_gb300/libmgg.so.  Re-running only recompiles units whose
sources or headers changed.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmgg.so")
HOST = os.path.join(PKG, "_host.so")  # the Python entry (csrc/host.cpp)
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmgg.so")


def _sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime() -> float:
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hdrs.append(os.path.join(INCLUDE, "mgg.h"))
    return max(os.path.getmtime(h) for h in hdrs)


def _compile(src: str, extra: list[str], verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, src[:-3] + ".o")
    srcp = os.path.join(CSRC, src)
    if os.path.exists(obj) and os.path.getmtime(obj) > max(os.path.getmtime(srcp), _deps_mtime()) \
            and not extra and not verbose_ptxas:
        return obj
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", srcp, "-o", obj]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas:
        sys.stderr.write(res.stderr)
    return obj


def _compile_host() -> str:
    """csrc/host.cpp against torch's headers -> _build/host-<torch>-<python>.o:
    an object is good for the versions that it was compiled against alone."""
    import sysconfig

    import torch
    versions = f"{torch.__version__}-{sysconfig.get_config_var('SOABI')}"
    src, obj = os.path.join(CSRC, "host.cpp"), os.path.join(BUILD, f"host-{versions}.o")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "mgg.h")))
    if os.path.exists(obj) and os.path.getmtime(obj) > newest:
        return obj
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(root, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *["-I" + i for i in inc], "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on host.cpp:\n{res.stdout}\n{res.stderr}")
    return obj


def _link_host(obj: str) -> str:
    """The extension module _host.so; it calls libmgg.so, found beside it."""
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = HOST + ".tmp"
    cmd = ["g++", "-shared", obj, "-o", tmp, "-L" + lib, "-Wl,-rpath," + lib, "-Wl,--no-as-needed",
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
           "-L" + PKG, "-l:libmgg.so", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, HOST)
    return HOST


def build_library(extra: list[str] | None = None, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    """Compile csrc/*.cu for sm_103a and link libmgg.so, then the Python entry
    _host.so over it; returns libmgg.so's path."""
    extra = list(extra or [])
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    jobs = jobs or min(len(srcs) + 1, os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        host = ex.submit(_compile_host)
        objs = list(ex.map(lambda s: _compile(s, extra, verbose_ptxas), srcs))
        host_obj = host.result()
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=libmgg.so", "-o", tmp,
           *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    _link_host(host_obj)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build_library(verbose_ptxas=v))
