"""In-tree build of the CUDA library (sm_103a only).

Each ``csrc/*.cu`` compiles to an object in parallel, then one shared library links them:
``top_gating_expert_gb300/libmoe_gb300.so``. nvcc cross-compiles without a GPU. Beside it,
``csrc/lists.cpp`` becomes the extension module ``_lists.so``, which reads lists of torch tensors. The library
needs neither torch nor Python's headers; the extension belongs to one version of both, and is built again by
itself when they or its sources change.
"""

from __future__ import annotations

import glob
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
LIBNAME = "libmoe_gb300.so"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def library_path() -> str:
    return os.path.join(PKG, LIBNAME)


def lists_path() -> str:
    return os.path.join(PKG, "_lists.so")


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the MoE library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(path: str, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(d) > os.path.getmtime(path) for d in deps)


def _needs_rebuild(lib: str) -> bool:
    return _older(lib, _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _lists_made_for() -> str:
    """What the extension is bound to: torch's version and Python's ABI."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def _lists_stamp() -> str:
    return os.path.join(BUILD, "lists.made_for")


def _lists_need_rebuild() -> bool:
    if _older(lists_path(), glob.glob(os.path.join(CSRC, "*.cpp")) + [os.path.join(INCLUDE, "moe.h"),
                                                                       os.path.abspath(__file__)]):
        return True
    try:
        with open(_lists_stamp()) as f:
            return f.read() != _lists_made_for()
    except (OSError, ImportError):  # without torch the build says so, after the library
        return True


def _build_lists(verbose: bool) -> None:
    import torch
    made_for = _lists_made_for()
    base = os.path.dirname(torch.__file__)
    tmp = lists_path() + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", f'-DBUILT_FOR="{torch.__version__}"',
           "-I", INCLUDE, "-I", os.path.join(base, "include"), "-I", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "lists.cpp"), "-o", tmp, "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu",
           "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on lists.cpp")
    os.replace(tmp, lists_path())
    with open(_lists_stamp(), "w") as f:
        f.write(made_for)


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link the library, and the extension, if any source is newer than them (the extension also for another
    torch or Python). Returns the library's path. Where the extension cannot be built the library is there all the
    same, and the error comes last."""
    lib = library_path()
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(1) as ex:
        lists = ex.submit(_build_lists, verbose) if force or _lists_need_rebuild() else None
        if force or _needs_rebuild(lib):
            _build_cuda(lib, verbose, extra_flags)
        if lists is not None:
            lists.result()
    return lib


def _build_cuda(lib: str, verbose: bool, extra_flags) -> None:
    nvcc = _nvcc()
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
        return obj

    with ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("linking the MoE library failed")
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
