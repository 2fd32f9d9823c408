"""Build libkvdecode.so (all CUDA sources, sm_103a) and the _binding module in-tree.

Each translation unit is compiled in parallel (nvcc; g++ for the CPython module, which is
written against PyTorch's C++ headers), then linked into one shared library and one module
next to this file. Intermediate objects go to ``_build/`` at the repo root.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkvdecode.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
BUILT_FOR = os.path.join(BUILD, "binding_torch")  # the PyTorch that _binding.so was compiled against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkvdecode.so")


def flags(ptxas_verbose: bool = False):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC, "-Xptxas",
                   "-v" if ptxas_verbose else "-O3"]


def _torch_dir() -> str:
    import importlib.util
    return os.path.dirname(importlib.util.find_spec("torch").origin)  # without importing it


def _torch_version() -> str:
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sys.version}\n{f.read()}"


def _torch_name() -> str:
    """torch.__version__, which the module carries and the package compares when it loads it."""
    return re.search(r"^__version__ = '([^']*)'", _torch_version(), re.M)[1]


def _compile(src: str, obj: str, verbose: bool) -> tuple[str, str]:
    if src.endswith(".cpp"):
        inc = os.path.join(_torch_dir(), "include")
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
        cmd = ["g++", "-c", src, "-o", obj, "-O2", "-std=c++17", "-fPIC",
               f'-DKVD_BUILT_FOR="{_torch_name()}"', "-I", INCLUDE,
               "-I", sysconfig.get_paths()["include"], "-isystem", inc, "-isystem",
               os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda]
    else:
        cmd = [nvcc(), "-c", src, "-o", obj] + flags(verbose)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return src, r.stderr


def _link_binding(obj: str) -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libkvdecode.so",
           "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
           "-lc10", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source and link libkvdecode.so and _binding.so (skipped when up
    to date and built for this PyTorch). Where the module cannot be built the library still is, and
    the error is raised behind it.
    `verbose` prints ptxas register / shared-memory / spill figures per kernel."""
    srcs = [BINDING_SRC] + sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = srcs + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(LIB) and os.path.exists(BINDING):
        lib_t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
        built_for = open(BUILT_FOR).read() if os.path.exists(BUILT_FOR) else ""
        if built_for == _torch_version() and all(os.path.getmtime(d) <= lib_t for d in deps):
            return LIB
    os.makedirs(BUILD, exist_ok=True)
    objs = [os.path.join(BUILD, os.path.splitext(os.path.basename(s))[0] + ".o")
            for s in srcs]
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        module = ex.submit(_compile, srcs[0], objs[0], verbose)
        for src, log in ex.map(lambda so: _compile(so[0], so[1], verbose), zip(srcs[1:], objs[1:])):
            if verbose and log:
                print(f"== {os.path.basename(src)}\n{log}", file=sys.stderr)
    tmp = LIB + f".tmp{os.getpid()}"
    # -z defs: an unresolved symbol fails the build here, not the first import on the GPU machine
    cmd = [nvcc(), "-shared", "-o", tmp] + objs[1:] + ARCH + ["-Xlinker", "-z", "-Xlinker", "defs"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    try:
        module.result()
        _link_binding(objs[0])
    except Exception:
        if os.path.exists(BINDING):  # one of an earlier library, with its calls
            os.remove(BINDING)
        raise
    with open(BUILT_FOR, "w") as f:
        f.write(_torch_version())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
