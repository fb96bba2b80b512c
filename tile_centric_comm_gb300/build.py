"""Build libtdg.so (the CUDA library behind include/tdg.h) in-tree for sm_103a.

    python -m tile_centric_comm_gb300.build [--force]

Each .cu under csrc/ is compiled in parallel with nvcc (one -gencode, sm_103a),
then linked into tile_centric_comm_gb300/_build/libtdg.so with the static CUDA
runtime, so the library has no load-time dependency on libcuda (the driver
entry points it needs are looked up at run time).  csrc/tdg_tensors.cpp,
the binding's tensor checks, becomes a CPython module beside it (g++, against
torch's headers).  The library needs neither torch nor that module: without
torch the module is left out, and when it does not compile the build warns.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libtdg.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtdg")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + [os.path.join(INCLUDE, "tdg.h")])


def _stale(target, inputs):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def tensors_path(torch_version: str) -> str:
    """The tensor checks' module for a version of torch and this Python: it
    reads their objects, so one built for others must not be loaded."""
    return os.path.join(BUILD, f"tdg_tensors.torch-{torch_version}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_tensors(force: bool = False) -> str | None:
    src = os.path.join(CSRC, "tdg_tensors.cpp")
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    torch = spec.submodule_search_locations[0]
    headers = os.path.join(torch, "include")
    version = os.path.join(torch, "version.py")
    target = tensors_path(runpy.run_path(version)["__version__"])
    if force or _stale(target, [src, version]):
        tmp = target + f".tmp{os.getpid()}"
        cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w", "-I", sysconfig.get_path("include"),
               "-I", headers, "-I", os.path.join(headers, "torch", "csrc", "api", "include"), src, "-o", tmp,
               "-L", os.path.join(torch, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for tdg_tensors.cpp:\n{r.stderr}")
        os.replace(tmp, target)
    return target


def _tensors_or_warning(force):
    try:
        build_tensors(force)
    except (OSError, RuntimeError) as e:
        warnings.warn(f"the binding's tensor checks were not built: {e}")


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    deps = _deps()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if not force and not _stale(LIB, srcs + deps):
        _tensors_or_warning(force)
        return LIB
    cc = nvcc()

    def compile_one(src_obj):
        src, obj = src_obj
        if not force and not _stale(obj, [src] + deps):
            return obj, ""
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        tensors = ex.submit(_tensors_or_warning, force)
        for obj, err in ex.map(compile_one, zip(srcs, objs)):
            if verbose and err:
                print(err, file=sys.stderr)
        tensors.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force=force, verbose=True, extra=extra))
