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


def _fingerprint(extra=()) -> str:
    h = hashlib.sha256()
    for p in sorted(glob.glob(os.path.join(CSRC, "*")) + [os.path.join(INCLUDE, "rowops.h")]):
        with open(p, "rb") as f:
            h.update(p.encode() + b"\0" + f.read())
    h.update(" ".join(ARCH + NVCC_FLAGS + list(extra)).encode())
    h.update(f"{importlib.metadata.version('torch')} {sys.version}".encode())
    return h.hexdigest()


def _host_command(out: str):
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    nvcc = os.path.realpath(_nvcc())
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    return [os.environ.get("CXX") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", f"-I{INCLUDE}",
            f"-I{torch}/include", f"-I{torch}/include/torch/csrc/api/include",
            f"-I{sysconfig.get_paths()['include']}", f"-I{cuda}", HOST_SOURCE, "-o", out, f"-L{torch}/lib",
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-ldl"]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link librowops.so if any source changed; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, "fingerprint")
    fp = _fingerprint(extra_flags)
    built = os.path.exists(LIB) and os.path.exists(HOST) and os.path.exists(stamp)
    if not force and built and open(stamp).read() == fp:
        return LIB
    nvcc = _nvcc()

    def compile_one(src):
        if src == HOST_SOURCE:
            r = subprocess.run(_host_command(host), capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"the C++ compiler failed on {os.path.basename(src)}:\n{r.stdout}{r.stderr}")
            return None
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

    host = HOST + f".tmp{os.getpid()}"
    srcs = [HOST_SOURCE, *_sources()]
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = [o for o in ex.map(compile_one, srcs) if o]
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)
    os.replace(host, HOST)
    with open(stamp, "w") as f:
        f.write(fp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
