"""Build libmoeroute.so in-tree with nvcc for sm_103a (GB300).

Each .cu translation unit compiles in its own nvcc process (in parallel),
then one nvcc link produces the shared library.  The CUDA runtime is linked
statically, so loading the library needs no GPU driver (only calls do).
The Python entry points of csrc/binding.cpp become _moe_ops.so beside it (g++,
torch's headers and libraries of the installation that runs the build).  Where
that fails, as with a torch without CUDA, the library is there all the same: a
warning says why, and only the calls that go through _moe_ops.so are missing.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libmoeroute.so")
OPS_PATH = os.path.join(OUT_DIR, "_moe_ops.so")
# what _moe_ops.so was built for: its layout of a tensor is torch's, its entry points are Python's
OPS_FOR_PATH = os.path.join(OUT_DIR, "_moe_ops.for")
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
        sorted(glob.glob(os.path.join(CSRC, "*.h"))) + [HEADER]


def _older(path, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(d) > os.path.getmtime(path) for d in deps)


def is_stale() -> bool:
    return _older(LIB_PATH, _deps())


def ops_for() -> str:
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def ops_built_for() -> str:
    """What ops_for() was when _moe_ops.so was built."""
    try:
        with open(OPS_FOR_PATH) as f:
            return f.read()
    except OSError:
        return "an unknown torch"


def ops_stale() -> bool:
    return ops_built_for() != ops_for() or _older(OPS_PATH, [BINDING, HEADER])


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r


def _compile_ops(nvcc):
    base = os.path.dirname(torch.__file__)
    obj = os.path.join(OUT_DIR, "binding.o")
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-c", BINDING, "-o", obj,
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          "-I", os.path.join(base, "include"),
          "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include"),
          "-I", sysconfig.get_paths()["include"]], f"g++ failed for {BINDING}")
    return obj


def _link_ops(obj):
    # torch's libraries are in the process when the module is imported; libmoeroute.so is
    # found beside it and is the copy that ctypes loads from the same path
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = OPS_PATH + f".{os.getpid()}.tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", torch_lib,
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", OUT_DIR, "-l:libmoeroute.so",
          "-Wl,-rpath,$ORIGIN"], "g++ link failed")
    os.replace(tmp, OPS_PATH)
    with open(OPS_FOR_PATH, "w") as f:
        f.write(ops_for())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile what is stale (or forced) and return the path of libmoeroute.so."""
    library, ops = force or is_stale(), force or ops_stale()
    if not library and not ops:
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = nvcc_path()
    flags = NVCC_FLAGS + (extra_flags or [])

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        r = _run([nvcc, *ARCH, *flags, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj],
                 f"nvcc failed for {src}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_ops, nvcc) if ops else None
        if library:
            objs = list(ex.map(compile_one, srcs))
            tmp = LIB_PATH + f".{os.getpid()}.tmp"
            _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], "nvcc link failed")
            os.replace(tmp, LIB_PATH)
    if ops:
        try:
            _link_ops(binding.result())
        except Exception as e:
            if os.path.exists(OPS_PATH):    # what an older build left there does not fit any more
                os.remove(OPS_PATH)
            warnings.warn(f"the Python entry points of {BINDING} were not built: {e}", RuntimeWarning,
                          stacklevel=2)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
