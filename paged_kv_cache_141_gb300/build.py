"""Build libpagedkv.so in-tree with nvcc for sm_103a (GB300), and with g++ the
binding's marshalling module _marshal.

Each CUDA translation unit compiles in its own nvcc process, in parallel;
the objects link into one shared library next to this file. The CUDA runtime
is linked statically, so the library loads without a GPU (the driver is only
opened by the first CUDA call). _marshal is compiled against this interpreter's
and the installed PyTorch's headers, under the interpreter's own suffix (no other
one imports it), and again when the PyTorch changes.

    python -m paged_kv_cache_141_gb300.build [--force] [-v]
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")
MARSHAL_SRC = os.path.join(PKG, "pysrc", "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    found = shutil.which("nvcc")
    if found:
        return found
    return os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _headers() -> list[str]:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(INCLUDE, "pagedkv.h"))
    return hs


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_marshal(force: bool = False) -> str:
    """The marshalling module, against this interpreter's and PyTorch's headers."""
    import torch
    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, os.path.basename(MARSHAL) + ".for")
    made_for = f"{sysconfig.get_config_var('SOABI')} {torch.__version__} {os.path.dirname(torch.__file__)}"
    try:
        with open(stamp) as f:
            same = f.read() == made_for
    except OSError:
        same = False
    if not force and same and not _stale(MARSHAL, [MARSHAL_SRC, os.path.join(INCLUDE, "pagedkv.h")]):
        return MARSHAL
    root = os.path.dirname(torch.__file__)
    libs = os.path.join(root, "lib")
    part = os.path.join(BUILD, f"_marshal.{os.getpid()}.so")    # moved into place when whole
    cmd = ["g++", "-O2", "-shared", "-fPIC", "-std=c++17", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I" + INCLUDE,
           "-isystem", os.path.join(root, "include"), "-I" + sysconfig.get_path("include"), MARSHAL_SRC,
           "-o", part, "-L" + libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath," + libs]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(MARSHAL_SRC)}:\n{proc.stderr}")
    os.replace(part, MARSHAL)
    with open(stamp, "w") as f:
        f.write(made_for)
    untagged = os.path.join(PKG, "_marshal.so")        # of an earlier build: any interpreter would import it
    if os.path.exists(untagged):
        os.remove(untagged)
    return MARSHAL


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(1) as side:
        marshal = side.submit(build_marshal, force)
        lib = _build_library(force, verbose)
        marshal.result()
    return lib


def _build_library(force: bool, verbose: bool) -> str:
    headers = _headers()
    jobs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        if force or _stale(obj, [src] + headers):
            jobs.append((src, obj))

    def compile_one(job):
        src, obj = job
        cmd = [nvcc()] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
        if verbose:
            cmd.append("-Xptxas=-v")
        proc = subprocess.run(cmd, capture_output=True, text=True)
        if proc.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{proc.stderr}")
        return proc.stderr

    if jobs:
        with ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
            for log in ex.map(compile_one, jobs):
                if verbose and log:
                    print(log)
    objs = [os.path.join(BUILD, os.path.splitext(os.path.basename(s))[0] + ".o") for s in sources()]
    if force or jobs or _stale(LIB, objs):
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", LIB] + objs
        subprocess.run(cmd, check=True)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
