"""Builds libpagedattn.so in-tree with nvcc for sm_103a.

Every .cu file under csrc/ is compiled in parallel (one -gencode, no other
architecture), then linked into ``_build/libpagedattn.so`` against the shared
CUDA runtime; ``_build/_pagedattn_calls.so`` is the Python side of the newer
calls. Re-running is cheap: nothing is rebuilt when the library is
newer than every source and header.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(BUILD, "libpagedattn.so")
ROOT = os.path.dirname(HERE)
BENCH_SRC = os.path.join(ROOT, "bench_loop.cpp")
BENCH_LIB = os.path.join(BUILD, "libpabench.so")

# The Python side of the newer calls (pa_python.cpp): a CPython module that
# reads torch tensors directly.
PYTHON_SRC = os.path.join(CSRC, "pa_python.cpp")
PYTHON_LIB = os.path.join(BUILD, "_pagedattn_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", "-cudart", "shared",
                     "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) +
            [PYTHON_SRC, os.path.abspath(__file__)])


def _python_built_for() -> str:
    """The torch and Python that _pagedattn_calls.so is compiled against, in a file
    beside it: their headers are not among the sources."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def up_to_date() -> bool:
    libs = (LIB, BENCH_LIB, PYTHON_LIB)
    if not all(os.path.exists(lib) for lib in libs):
        return False
    try:
        with open(PYTHON_LIB + ".for") as f:
            if f.read() != _python_built_for():
                return False
    except OSError:
        return False
    t = min(os.path.getmtime(lib) for lib in libs)
    return all(os.path.getmtime(p) <= t for p in _deps() + [BENCH_SRC])


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link; returns the library path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or ptxas_info or r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
        return obj

    def compile_python() -> str:
        import sysconfig
        import torch
        root = os.path.dirname(torch.__file__)
        obj = os.path.join(BUILD, "pa_python.o")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE,
               "-I", sysconfig.get_paths()["include"],
               "-I", os.path.join(root, "include"),
               "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
               "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
               "-c", PYTHON_SRC, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError("compiling pa_python.cpp failed")
        return obj

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=max(2, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        python_obj = ex.submit(compile_python)
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-Xlinker", "-soname=libpagedattn.so", "-Xlinker", "-rpath=/usr/local/cuda/lib64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc link failed")
    os.replace(tmp, LIB)
    # The benchmark's native step loops (bench_loop.cpp, beside bench.py):
    # host code only, linked against the library above.
    if os.path.exists(BENCH_SRC):
        tmp = BENCH_LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, "-shared", "-std=c++17", "-O2", "-Xcompiler", "-fPIC", "-cudart", "shared",
               "-I", ROOT, BENCH_SRC, "-o", tmp, "-L", BUILD, "-lpagedattn",
               "-Xlinker", "-rpath=$ORIGIN", "-Xlinker", "-rpath=/usr/local/cuda/lib64"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("bench loop build failed")
        os.replace(tmp, BENCH_LIB)
    # Last: what it lacks (torch's headers, a compiler that takes them) keeps nothing
    # else from being built.
    import torch
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = PYTHON_LIB + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, python_obj.result(), "-L", BUILD, "-lpagedattn", "-L", torch_lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN",
           f"-Wl,-rpath,{torch_lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("linking _pagedattn_calls failed")
    os.replace(tmp, PYTHON_LIB)
    with open(PYTHON_LIB + ".for", "w") as f:
        f.write(_python_built_for())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
