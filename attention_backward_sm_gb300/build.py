"""Builds libfabwd.so in-tree for sm_103a with nvcc (no cmake), and the host
extension _paged_host.so beside it with g++ against the installed PyTorch.

Each translation unit compiles to an object in parallel, then nvcc links
the shared library next to this file.  A rebuild happens only when a
source or header is newer than the library (the extension: also when PyTorch
or Python changed).  The library needs neither; without a PyTorch that has
CUDA it is all that is built.
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
HEADERS = ["internal.h", "sm103.cuh", "paged.h", "decode.cuh", "decode_shape.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _torch_dir() -> str | None:
    """The folder of the installed PyTorch, None without one that has CUDA."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    path = spec.submodule_search_locations[0]
    return path if os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def _host_needs() -> str:
    """What HOST is built against: this PyTorch and this Python."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f.read() + str(sysconfig.get_config_var("EXT_SUFFIX"))


def _host_tag() -> str:
    try:
        with open(HOST_TAG) as f:
            return f.read()
    except OSError:
        return ""


def _older(path: str, sources) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    deps = [os.path.join(CSRC, f) for f in sources]
    deps += [os.path.join(ROOT, "include", "fabwd.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _compile_host() -> str:
    obj = os.path.join(BUILD, HOST_SOURCE.replace(".cpp", ".o"))
    inc = [os.path.join(_torch_dir(), "include"), os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           sysconfig.get_paths()["include"]]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", *[a for i in inc for a in ("-isystem", i)], "-c",
          os.path.join(CSRC, HOST_SOURCE), "-o", obj], f"g++ for {HOST_SOURCE}")
    return obj


def _link_host(obj: str) -> None:
    tmp = HOST + ".tmp"
    libs = os.path.join(_torch_dir(), "lib")
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + os.path.dirname(LIB), "-l:" + os.path.basename(LIB), "-L" + libs,
          "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN",
          "-Wl,-rpath," + libs], "g++ link")
    os.replace(tmp, HOST)
    with open(HOST_TAG, "w") as f:
        f.write(_host_needs())


def build(force: bool = False, verbose: bool = False) -> str:
    make_lib = force or _older(LIB, SOURCES + HEADERS)
    make_host = _torch_dir() is not None and (force or _host_tag() != _host_needs() or _older(HOST, [HOST_SOURCE]))
    if not make_lib and not make_host:
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        out = _run(cmd, f"nvcc for {src}")
        if verbose and out:
            sys.stderr.write(out)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        host_obj = ex.submit(_compile_host) if make_host else None
        if make_lib:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + ".tmp"
            _run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], "nvcc link")
            os.replace(tmp, LIB)
        if make_host:   # a failure here leaves the library in place
            _link_host(host_obj.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
