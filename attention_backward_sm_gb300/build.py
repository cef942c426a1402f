"""Builds libfabwd.so in-tree for sm_103a with nvcc (no cmake), and the host
extension _paged_host.so beside it with g++ against the installed PyTorch.

Each translation unit compiles to an object in parallel, then nvcc links
the shared library next to this file.  A rebuild happens only when a
source or header is newer than the library, or when PyTorch changed.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libfabwd.so")
HOST = os.path.join(HERE, "_paged_host.so")
HOST_SOURCE = "paged_host.cpp"
HOST_TAG = os.path.join(BUILD, "host_torch")   # the PyTorch that HOST was built against
SOURCES = ["api.cu", "small_kernels.cu", "fwd_main.cu", "bwd_main.cu", "bwd_d256.cu", "dq_main.cu", "noalloc.cu",
           "paged.cu", "decode.cu", "decode_d64.cu", "decode_d128.cu", "decode_d256.cu"]
HEADERS = ["internal.h", "sm103.cuh", "paged.h", "decode.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _torch_version() -> str:
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f.read()


def _host_tag() -> str:
    try:
        with open(HOST_TAG) as f:
            return f.read()
    except OSError:
        return ""


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(HOST) or _host_tag() != _torch_version():
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(HOST))
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + [HOST_SOURCE]]
    deps.append(os.path.join(ROOT, "include", "fabwd.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    def compile_host():
        obj = os.path.join(BUILD, HOST_SOURCE.replace(".cpp", ".o"))
        inc = [os.path.join(_torch_dir(), "include"), os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
               sysconfig.get_paths()["include"]]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", *[a for i in inc for a in ("-isystem", i)], "-c",
               os.path.join(CSRC, HOST_SOURCE), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {HOST_SOURCE}:\n{r.stdout}\n{r.stderr}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        host_obj = ex.submit(compile_host)
        objs = list(ex.map(compile_one, SOURCES))
        host_obj = host_obj.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = HOST + ".tmp"
    libs = os.path.join(_torch_dir(), "lib")
    cmd = ["g++", "-shared", "-o", tmp, host_obj, "-L" + HERE, "-l:" + os.path.basename(LIB), "-L" + libs, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, HOST)
    with open(HOST_TAG, "w") as f:
        f.write(_torch_version())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
