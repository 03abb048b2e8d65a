"""Build libpa.so (the CUDA kernels and their C ABI) in-tree with nvcc, and
_native.so, the Python binding of some of its calls, with the host compiler
against the installed PyTorch.

    python -m paged_kv_cache_226_gb300.build [--force]

One ``-gencode`` (sm_103a), translation units compiled in parallel, the CUDA
runtime linked statically so the library needs no libcuda at load time.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libpa.so")
# csrc/binding.cpp, compiled
BINDING = os.path.join(CSRC, "binding.cpp")
NATIVE_PATH = os.path.join(PKG, "_native.so")
# the same sources with the failure-detection test hooks (include/pa_test.h)
TEST_BUILD_DIR = os.path.join(PKG, "_build_test")
TEST_LIB_PATH = os.path.join(PKG, "libpa_test.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--cudart", "static",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + \
        [os.path.abspath(__file__)]


def up_to_date(lib_path: str = LIB_PATH) -> bool:
    if not os.path.exists(lib_path):
        return False
    t = os.path.getmtime(lib_path)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _native_stamp() -> str:
    """What _native.so depends on besides its source."""
    import torch
    return f"{torch.__version__} {torch.__path__[0]} {sys.version}"


def native_up_to_date() -> bool:
    stamp = os.path.join(BUILD_DIR, "native.stamp")
    if not (os.path.exists(NATIVE_PATH) and os.path.exists(stamp)):
        return False
    with open(stamp) as f:
        if f.read() != _native_stamp():
            return False
    t = os.path.getmtime(NATIVE_PATH)
    return all(os.path.getmtime(p) <= t
               for p in [BINDING, os.path.join(INCLUDE, "pa.h"), os.path.abspath(__file__)])


def _compile_native() -> str:
    """binding.cpp to an object file."""
    import torch
    inc = os.path.join(torch.__path__[0], "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    obj = os.path.join(BUILD_DIR, "binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
           os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-c", BINDING, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_native(obj: str) -> None:
    import torch
    tmp = NATIVE_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", os.path.join(torch.__path__[0], "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE_PATH)
    with open(os.path.join(BUILD_DIR, "native.stamp"), "w") as f:
        f.write(_native_stamp())


def build(force: bool = False, verbose: bool = False, extra_flags=(),
          test_hooks: bool = False) -> str:
    """Build libpa.so and _native.so (or, with test_hooks, libpa_test.so: the
    CUDA sources compiled with -DPA_TEST_HOOKS) and return the library's path."""
    lib_path = TEST_LIB_PATH if test_hooks else LIB_PATH
    build_dir = TEST_BUILD_DIR if test_hooks else BUILD_DIR
    if test_hooks:
        extra_flags = (*extra_flags, "-DPA_TEST_HOOKS=1")
    kernels = force or not up_to_date(lib_path)
    native = not test_hooks and (force or not native_up_to_date())
    if not kernels and not native:
        return lib_path
    nvcc = _nvcc()
    os.makedirs(build_dir, exist_ok=True)
    objs = []

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_native) if native else None
        objs = list(ex.map(compile_one, sources())) if kernels else []
    if kernels:
        _link(nvcc, lib_path, objs)
    if native:
        _link_native(binding.result())
    return lib_path


def _link(nvcc: str, lib_path: str, objs) -> None:
    tmp = lib_path + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "--cudart", "static", "-Xlinker",
           f"-soname={os.path.basename(lib_path)}", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills")
    a = ap.parse_args()
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info,
                extra_flags=extra))
