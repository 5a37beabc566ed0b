"""Builds the layer's shared library in-tree: _build/libwse.so (sm_103a).

Each .cu file is compiled in parallel with nvcc, then linked into one shared
library against the shared CUDA runtime.  Beside it the Python extension module
of the attention and sampling calls, _build/wse_calls.so, is compiled with g++
and linked against that library and PyTorch's; the library needs neither, and is
built also where the module cannot be.  Rebuilds only what is older than its
sources and headers.

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


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def _library_inputs():
    return _sources() + [p for end in ("*.cuh", "*.h") for p in glob.glob(os.path.join(CSRC, end))] + _headers()


def _inputs():
    return _library_inputs() + [CALLS_SOURCE]


def _newer(path: str, inputs) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in inputs)


def _library_up_to_date() -> bool:
    return _newer(LIB, _library_inputs())


def _calls_up_to_date() -> bool:
    return _newer(CALLS, [CALLS_SOURCE] + _headers())


def up_to_date() -> bool:
    return _library_up_to_date() and _calls_up_to_date()


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")  # found, not imported: the headers are all that is wanted
    return spec.submodule_search_locations[0] if spec is not None and spec.submodule_search_locations else None


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


def _link_calls(obj: str):
    tmp = CALLS + f".tmp{os.getpid()}"
    torch_lib = os.path.join(_torch_dir(), "lib")
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{BUILD}", "-lwse", "-Wl,-rpath,$ORIGIN", f"-L{torch_lib}",
          "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{torch_lib}"], "link of the Python calls")
    os.replace(tmp, CALLS)


def build_library(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """The C library alone."""
    if not force and _library_up_to_date():
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

    with ThreadPoolExecutor(max_workers=jobs or min(len(srcs), max(4, os.cpu_count() or 8))) as ex:
        results = list(ex.map(compile_one, srcs))
    for src, (_, log) in zip(srcs, results):
        if verbose or "warning" in log:  # compiler warnings are shown, not swallowed
            sys.stderr.write(f"{os.path.basename(src)}:\n{log}")
    tmp = LIB + f".tmp{os.getpid()}"
    _run([cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp] + [o for o, _ in results], "link")
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """The library and the module of the Python calls.  Without PyTorch the
    module is left out, with a note; what else keeps it from being built is
    raised once the library is in place."""
    if not force and _calls_up_to_date():
        return build_library(verbose=verbose, jobs=jobs)
    if _torch_dir() is None:
        path = build_library(force, verbose, jobs)
        sys.stderr.write("PyTorch not found: the module of the attention and sampling calls is not built\n")
        return path
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        calls = ex.submit(_compile_calls)  # beside the kernels
        path = build_library(force, verbose, jobs)
        _link_calls(calls.result())
    return path


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
