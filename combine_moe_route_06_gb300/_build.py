"""Build libmoeroute.so in-tree with nvcc for sm_103a (GB300).

Each .cu translation unit compiles in its own nvcc process (in parallel),
then one nvcc link produces the shared library.  The CUDA runtime is linked
statically, so loading the library needs no GPU driver (only calls do).
The Python entry points of csrc/binding.cpp become _moe_ops.so beside it (g++,
torch's headers and libraries of the installation that runs the build).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libmoeroute.so")
OPS_PATH = os.path.join(OUT_DIR, "_moe_ops.so")
BINDING = os.path.join(CSRC, "binding.cpp")
HEADER = os.path.join(ROOT, "include", "moe_route.h")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-Xptxas", "-warn-spills", "--expt-relaxed-constexpr"]


def nvcc_path() -> str:
    for cand in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        p = os.path.join(cand, "bin", "nvcc") if cand else ""
        if p and os.path.exists(p):
            return p
    p = shutil.which("nvcc")
    if not p:
        raise RuntimeError("nvcc not found: set CUDA_HOME or put nvcc on PATH")
    return p


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.h"))) + [BINDING, HEADER]


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(OPS_PATH):
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(OPS_PATH))
    return any(os.path.getmtime(d) > t for d in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile (if stale or forced) and return the path of libmoeroute.so."""
    if not force and not is_stale():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = nvcc_path()
    flags = NVCC_FLAGS + (extra_flags or [])
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *flags, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    def compile_binding():
        base = os.path.dirname(torch.__file__)
        obj = os.path.join(OUT_DIR, "binding.o")
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-c", BINDING, "-o", obj,
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
               "-I", os.path.join(base, "include"),
               "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include"),
               "-I", sysconfig.get_paths()["include"]]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {BINDING}:\n{r.stdout}\n{r.stderr}")
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, srcs))
        binding_obj = binding.result()
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    # torch's libraries are in the process when the module is imported; libmoeroute.so is
    # found beside it and is the copy that ctypes loads from the same path
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = OPS_PATH + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, binding_obj, "-L", torch_lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", OUT_DIR, "-l:libmoeroute.so",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OPS_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
