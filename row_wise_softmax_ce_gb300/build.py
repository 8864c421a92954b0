"""Build the CUDA library ``libcerows.so`` in-tree with nvcc, for sm_103a only,
and the objectives' PyTorch binding ``_binding.so`` beside it with g++.

Each translation unit compiles in parallel; the objects are then linked into
one shared library with the CUDA runtime linked statically, so the library
needs no CUDA shared library of its own beyond the driver. The binding links to
it and to PyTorch's libraries, which are loaded before it.

    python -m row_wise_softmax_ce_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
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
LIB = os.path.join(PKG, "libcerows.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_FOR = os.path.join(BUILD, "binding_for.txt")  # what the binding was built against

SOURCES = ["ce_kernels.cu", "ce_objectives.cu", "ce_choices.cu", "ce_router.cu", "ce_api.cu"]
HEADERS = ["ce_device.cuh", "ce_objectives.cuh", "ce_internal.h", "ce_launch.h"]
BINDING_SOURCE = "binding.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _inputs() -> list[str]:
    return ([os.path.join(CSRC, s) for s in SOURCES + HEADERS + [BINDING_SOURCE]]
            + [os.path.join(INCLUDE, "ce_rows.h"), os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    if _read(BINDING_FOR) != _binding_for():
        return False  # another PyTorch or Python since
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _run(cmd: list[str], verbose: bool, what: str) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 or verbose:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {what}")


def _torch_dir() -> str:
    return list(importlib.util.find_spec("torch").submodule_search_locations)[0]


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def _binding_for() -> str:
    """The Python ABI and the PyTorch (where it is, and its version file) that a binding fits."""
    torch = _torch_dir()
    return "\n".join([sysconfig.get_config_var("SOABI") or "", torch, _read(os.path.join(torch, "version.py"))])


def _compile_binding(cc: str, verbose: bool) -> str:
    torch = _torch_dir()
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")
    obj = os.path.join(BUILD, "binding.o")
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-I{INCLUDE}",
          f"-I{torch}/include", f"-I{torch}/include/torch/csrc/api/include", f"-I{cuda}",
          f"-I{sysconfig.get_paths()['include']}", "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj], verbose,
         BINDING_SOURCE)
    return obj


def _link_binding(obj: str, verbose: bool) -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    libs = ["torch_python", "torch", "torch_cpu", "torch_cuda", "c10", "c10_cuda"]
    _run([os.environ.get("CXX", "g++"), "-shared", obj, "-o", tmp, f"-L{_torch_dir()}/lib", *[f"-l{n}" for n in libs],
          f"-L{PKG}", "-l:libcerows.so", "-Wl,-rpath,$ORIGIN", "-Wl,-z,now"], verbose, "the binding")
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(_binding_for())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link; returns the library path. Rebuilds only when a
    source is newer than the library or the binding was built against another
    PyTorch or Python (or ``force``)."""
    if not force and not ptxas_info and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or (verbose or ptxas_info):
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}")
        return obj

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, cc, verbose)
        objs = list(ex.map(compile_one, SOURCES))
        binding_obj = binding.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    _link_binding(binding_obj, verbose)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills/shared memory")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))
