"""Builds librowops.so (the CUDA kernels and the C ABI) in-tree for sm_103a.

Each .cu file is compiled in its own nvcc process (in parallel) and the
objects are linked into ``row_wise_softmax_warp_gb300/librowops.so`` with the
CUDA runtime linked statically.  Only one architecture is generated:
``-gencode arch=compute_103a,code=sm_103a``.  Beside them the C++ compiler makes
``_host.so``, the compiled part of the Python binding, against the installed torch.
"""
from __future__ import annotations

import glob
import hashlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librowops.so")
HOST_SOURCE = os.path.join(CSRC, "host_binding.cpp")
HOST = os.path.join(PKG, "_host.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit's bin/ on PATH")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _digest(paths, *rest) -> str:
    h = hashlib.sha256()
    for p in sorted(paths):
        with open(p, "rb") as f:
            h.update(p.encode() + b"\0" + f.read())
    h.update(" ".join(rest).encode())
    return h.hexdigest()


def _fingerprint(extra=()) -> str:
    sources = set(glob.glob(os.path.join(CSRC, "*"))) - {HOST_SOURCE}
    return _digest([*sources, os.path.join(INCLUDE, "rowops.h")], *ARCH, *NVCC_FLAGS, *extra)


def _current(stamp: str, out: str, fingerprint: str) -> bool:
    if not os.path.exists(out) or not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read() == fingerprint


def _stamp(stamp: str, fingerprint: str) -> None:
    with open(stamp, "w") as f:
        f.write(fingerprint)


def _host_command(out: str):
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    nvcc = os.path.realpath(_nvcc())
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    return [os.environ.get("CXX") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", f"-I{INCLUDE}",
            f"-I{torch}/include", f"-I{torch}/include/torch/csrc/api/include",
            f"-I{sysconfig.get_paths()['include']}", f"-I{cuda}", HOST_SOURCE, "-o", out, f"-L{torch}/lib",
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-ldl"]


def _build_host(force: bool) -> None:
    """Compile _host.so if its source, the C ABI, torch or Python changed."""
    stamp = os.path.join(BUILD, "fingerprint_host")
    fp = _digest([HOST_SOURCE, os.path.join(INCLUDE, "rowops.h")], *_host_command(HOST), sys.version,
                 importlib.metadata.version("torch"))
    if not force and _current(stamp, HOST, fp):
        return
    tmp = HOST + f".tmp{os.getpid()}"
    r = subprocess.run(_host_command(tmp), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the C++ compiler failed on {os.path.basename(HOST_SOURCE)}:\n{r.stdout}{r.stderr}")
    os.replace(tmp, HOST)
    _stamp(stamp, fp)


def _build_library(ex, force: bool, verbose: bool, extra_flags) -> None:
    stamp = os.path.join(BUILD, "fingerprint")
    fp = _fingerprint(extra_flags)
    if not force and _current(stamp, LIB, fp):
        return
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)
    _stamp(stamp, fp)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link librowops.so if any source changed; returns its path.

    _host.so is compiled beside it.  The library and the operators that are called by
    ctypes do without: where it cannot be compiled (no headers of Python, another torch), a
    warning says why, and the calls that need it raise.
    """
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=max(1, min(len(_sources()) + 1, os.cpu_count() or 1))) as ex:
        host = ex.submit(_build_host, force)
        _build_library(ex, force, verbose, extra_flags)
        try:
            host.result()
        except Exception as e:  # noqa: BLE001 - whatever it lacks, the library is there
            if os.path.exists(HOST):
                os.remove(HOST)  # made for other sources or another torch
            warnings.warn(f"the compiled part of the Python binding (_host.so) was not built: {e}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
