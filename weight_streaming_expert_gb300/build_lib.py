"""Builds the layer's shared library in-tree: _build/libwse.so (sm_103a).

Each .cu file is compiled in parallel with nvcc, then linked into one shared
library against the shared CUDA runtime.  The Python extension module of the
attention and sampling calls, _build/wse_calls.so, is compiled beside them
with g++ and linked against that library and PyTorch's.  Rebuilds only when a
source or header is newer than the libraries.

    python -m weight_streaming_expert_gb300.build_lib [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libwse.so")
CALLS = os.path.join(BUILD, "wse_calls.so")
CALLS_SOURCE = os.path.join(CSRC, "python_calls.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                     "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return (_sources() + [CALLS_SOURCE] + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALLS):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")  # found, not imported: the headers are all that is wanted
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch not found: the Python calls are compiled against its headers")
    return spec.submodule_search_locations[0]


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_calls() -> str:
    obj = os.path.join(BUILD, "python_calls.o")
    torch_include = os.path.join(_torch_dir(), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-c", CALLS_SOURCE, "-o", obj, "-I", INCLUDE, "-isystem", torch_include,
          "-isystem", os.path.join(torch_include, "torch", "csrc", "api", "include"), "-isystem",
          sysconfig.get_paths()["include"]], "g++ on python_calls.cpp")
    return obj


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, (r.stdout + r.stderr)

    with ThreadPoolExecutor(max_workers=jobs or min(len(srcs) + 1, max(4, os.cpu_count() or 8))) as ex:
        calls = ex.submit(_compile_calls)
        results = list(ex.map(compile_one, srcs))
        calls_obj = calls.result()
    for src, (_, log) in zip(srcs, results):
        if verbose or "warning" in log:  # compiler warnings are shown, not swallowed
            sys.stderr.write(f"{os.path.basename(src)}:\n{log}")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = CALLS + f".tmp{os.getpid()}"
    torch_lib = os.path.join(_torch_dir(), "lib")
    _run(["g++", "-shared", "-o", tmp, calls_obj, f"-L{BUILD}", "-lwse", "-Wl,-rpath,$ORIGIN", f"-L{torch_lib}",
          "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{torch_lib}"], "link of the Python calls")
    os.replace(tmp, CALLS)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
