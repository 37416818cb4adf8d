"""Builds libswin_wattn.so in-tree with nvcc for sm_103a.

Each CUDA source is compiled to an object in parallel, then linked into a
shared library beside this file; the binding's argument checks (arguments.cpp)
become a module of their own there, for this Python and this PyTorch only.  No
CMake, no torch extension machinery.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libswin_wattn.so")
ARGUMENTS = os.path.join(HERE, "_arguments" + sysconfig.get_config_var("EXT_SUFFIX"))
ARGUMENTS_TORCH = os.path.join(BUILD, "arguments.torch")   # the PyTorch that ARGUMENTS was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer(built, files):
    return os.path.exists(built) and os.path.getmtime(built) >= max(os.path.getmtime(f) for f in files)


def _library_current():
    inc = os.path.join(ROOT, "include")
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return _newer(LIB, files + [os.path.join(inc, f) for f in os.listdir(inc)] + [os.path.abspath(__file__)])


def _torch_dir():
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def torch_version() -> str:
    """torch.__version__, without importing it."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return re.search(r"^__version__ = ['\"](.+)['\"]", f.read(), re.M).group(1)


def arguments_current() -> bool:
    """Whether the argument checks are built, from these sources and for this PyTorch
    (their file's name holds the Python)."""
    if not _newer(ARGUMENTS, [os.path.join(CSRC, "arguments.cpp"), os.path.abspath(__file__)]):
        return False
    try:
        with open(ARGUMENTS_TORCH) as f:
            return f.read() == torch_version()
    except OSError:
        return False


def _build_arguments():
    torch, version = _torch_dir(), torch_version()
    tmp = ARGUMENTS + ".%d.tmp" % os.getpid()
    res = subprocess.run(
        ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", '-DTORCH_BUILT="%s"' % version, "-I", sysconfig.get_paths()["include"],
         "-I", os.path.join(torch, "include"), "-I", os.path.join(torch, "include/torch/csrc/api/include"),
         os.path.join(CSRC, "arguments.cpp"), "-o", tmp, "-L", os.path.join(torch, "lib"), "-ltorch_cpu", "-lc10"],
        capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(res.stdout + res.stderr)
    os.replace(tmp, ARGUMENTS)
    os.makedirs(BUILD, exist_ok=True)
    with open(ARGUMENTS_TORCH, "w") as f:
        f.write(version)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        beside = ex.submit(_build_arguments) if force or not arguments_current() else None
        if force or not _library_current():
            _build_library(verbose, extra_flags)
        try:
            if beside:
                beside.result()
        except Exception as e:   # (the library works without: the binding's Python checks do)
            sys.stderr.write("arguments.cpp is not built, calls on few rows take longer: %s\n" % e)
    return LIB


def _build_library(verbose, extra_flags):
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, res.stdout, res.stderr))
        if verbose and (res.stdout or res.stderr):
            sys.stderr.write(res.stdout + res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".%d.tmp" % os.getpid()
    res = subprocess.run([cc, *ARCH, "-shared", "-cudart", "shared", *objs, "-o", tmp], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
