"""Builds libidx.so (the C ABI of the indexer) in-tree with nvcc for sm_103a,
and the host extension of the latent calls.

The translation units are compiled in parallel and linked into
``sparse_attention_indexer_mxfp4_gb300/_build/libidx.so``, which needs nvcc
alone.  The extension also needs torch's and Python's headers; its file, beside
the library, is named by the torch and the Python it was built for.  Each is
rebuilt only when a source or header of its own is newer.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from importlib import metadata
from importlib.util import find_spec

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libidx.so")


def _torch_version() -> str:
    try:
        return metadata.version("torch")
    except metadata.PackageNotFoundError:
        return ""


CALLS = os.path.join(BUILD, f"_latent_calls-torch{_torch_version()}{sysconfig.get_config_var('EXT_SUFFIX')}")
CALLS_SRC = os.path.join(CSRC, "bind_latent.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the indexer library cannot be built")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(ROOT, "include", "idx.h")])


def _newer(made: str, inputs: list[str]) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(p) <= os.path.getmtime(made) for p in inputs)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def calls_up_to_date() -> bool:
    return _newer(CALLS, [CALLS_SRC, os.path.join(ROOT, "include", "idx.h")])


def _calls_command(out: str) -> list[str]:
    torch = os.path.dirname(find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"],
               os.path.join(torch, "include"), os.path.join(cuda, "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", *(f"-I{i}" for i in include), CALLS_SRC,
            "-o", out, "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_cuda", "-ltorch_python"]


def _start(src: str, cmd: list[str]):
    return src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _failed(procs, verbose: bool) -> list[str]:
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stdout.write(out)
        if p.returncode != 0:
            failed.append(src)
    return failed


def build_library(force: bool = False, verbose: bool = False) -> str:
    """libidx.so."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        procs.append(_start(src, [nvcc, *ARCH, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src,
                                  "-o", obj]))
    failed = _failed(procs, verbose)
    if failed:
        raise RuntimeError(f"nvcc failed on {failed}")
    tmp = LIB + f".{os.getpid()}.tmp"
    subprocess.check_call([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


def _start_calls(force: bool):
    """The extension's compiler at work on a file of its own, or None."""
    if not force and calls_up_to_date():
        return None
    os.makedirs(BUILD, exist_ok=True)
    tmp = CALLS + f".{os.getpid()}.tmp"
    return tmp, [_start(CALLS_SRC, _calls_command(tmp))]


def _finish_calls(started, verbose: bool) -> str:
    if started is not None:
        tmp, procs = started
        if _failed(procs, verbose):
            raise RuntimeError(f"the compiler failed on {CALLS_SRC}")
        os.replace(tmp, CALLS)
    return CALLS


def build_calls(force: bool = False, verbose: bool = False) -> str:
    """The latent calls' extension."""
    return _finish_calls(_start_calls(force), verbose)


def build(force: bool = False, verbose: bool = False) -> str:
    """Both, side by side; the library is there although the extension fails."""
    calls = _start_calls(force)
    try:
        build_library(force, verbose)
    finally:
        _finish_calls(calls, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
