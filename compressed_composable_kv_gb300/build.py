"""In-tree build of libc2kv.so for sm_103a (nvcc, no cmake).

Each CUDA translation unit is compiled in parallel, then linked into one
shared library with the CUDA runtime linked statically.  The binding's
marshalling module (_marshal.so, C++ against torch's headers) is built beside
it.  The results live in compressed_composable_kv_gb300/_build/ (git-ignored).
"""
from __future__ import annotations

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
LIB = os.path.join(BUILD, "libc2kv.so")
MARSHAL = os.path.join(BUILD, "_marshal.so")

SOURCES = ["api.cu", "rope.cu", "attn.cu", "prefill_tc.cu", "decode_tc.cu", "linear_tc.cu",
           "api_pages8.cu", "pages8.cu", "attend_pages8.cu", "logprobs.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the C2KV CUDA library cannot be built")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-I", INCLUDE, "-I", CSRC] + list(extra)


def _fresh(target: str, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in deps)


def _lib_fresh() -> bool:
    files = [os.path.join(CSRC, f) for f in SOURCES + [f for f in os.listdir(CSRC) if f.endswith(".h")]]
    return _fresh(LIB, files + [os.path.join(INCLUDE, "c2kv.h"), os.path.abspath(__file__)])


def _marshal_fresh() -> bool:
    return marshal_fits_torch() and _fresh(MARSHAL, [os.path.join(CSRC, "marshal.cpp"), os.path.join(INCLUDE, "c2kv.h"),
                                                     os.path.abspath(__file__)])


def _torch_tag() -> str:
    """What _marshal.so is bound to: this torch, by place and version, and this Python."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return "\n".join([_torch_dir(), sys.implementation.cache_tag, f.read()])


def marshal_fits_torch() -> bool:
    """Whether _marshal.so was built for the torch and Python that run."""
    try:
        with open(MARSHAL + ".torch") as f:
            return f.read() == _torch_tag()
    except OSError:
        return False


def up_to_date() -> bool:
    return _lib_fresh() and _marshal_fresh()


def _torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _run(cmd):
    try:
        return subprocess.run(cmd, capture_output=True, text=True)
    except FileNotFoundError as e:
        return subprocess.CompletedProcess(cmd, 1, "", f"{e}\n")


def _compile_marshal():
    """marshal.cpp to an object; it is linked once libc2kv.so is there."""
    inc = os.path.join(_torch_dir(), "include")
    return _run(["g++", "-O2", "-std=c++20", "-fPIC", "-I", INCLUDE, "-isystem", inc, "-isystem",
                 os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"],
                 "-c", os.path.join(CSRC, "marshal.cpp"), "-o", os.path.join(BUILD, "marshal.o")])


def _link_marshal():
    lib = os.path.join(_torch_dir(), "lib")
    r = _run(["g++", "-shared", "-o", MARSHAL + ".tmp", os.path.join(BUILD, "marshal.o"), LIB, "-L", lib,
              "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])
    if r.returncode == 0:
        if os.path.exists(MARSHAL + ".torch"):   # no tag while it may be another module's
            os.remove(MARSHAL + ".torch")
        os.replace(MARSHAL + ".tmp", MARSHAL)
        with open(MARSHAL + ".torch", "w") as f:
            f.write(_torch_tag())
    return r


def _build_lib(verbose: bool, extra) -> None:
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc] + _flags(extra) + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    for src, _, r in results:
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}")
    tmp = LIB + ".tmp"
    cmd = [cc] + ARCH + ["-shared", "-Xlinker", "-soname=libc2kv.so", "-o", tmp] + [o for _, o, _ in results] + ["-lcuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        # libcuda.so may be absent on a build host without a driver; the
        # library only needs it through the runtime, so link without it.
        cmd = cmd[:-1]
        r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("linking libc2kv.so failed")
    os.replace(tmp, LIB)


def build_library(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile what is missing or stale; return libc2kv.so's path.  Where
    _marshal.so cannot be built (no g++ with C++20, no torch headers) the
    compiler's message is shown and libc2kv.so is built all the same: only the
    calls that go by way of that module raise ImportError."""
    lib, marshal = force or not _lib_fresh(), force or not _marshal_fresh()
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        compiled = ex.submit(_compile_marshal) if marshal else None
        if lib:
            _build_lib(verbose or ptxas_verbose, ["-Xptxas", "-v"] if ptxas_verbose else [])
    if marshal:
        r = compiled.result()
        if r.returncode == 0:
            r = _link_marshal()
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr + "_marshal.so is not built\n")
            if os.path.exists(MARSHAL):   # of older sources
                os.remove(MARSHAL)
    return LIB


if __name__ == "__main__":
    build_library(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv)
    print(LIB)
