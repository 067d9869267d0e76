"""Build libattnprefill.so in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` compiles to an object in parallel, then nvcc links the
shared library (CUDA runtime linked statically), and g++ the small CPython
extension that marshals the serving-step calls to it. Run as a module
(``python -m chunked_prefill_gqa_gb300.build``) or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libattnprefill.so")
BINDING = os.path.join(OUT, "_binding.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def _nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattnprefill.so")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(glob.glob(os.path.join(CSRC, "*.cpp"))) + \
        [os.path.join(INCLUDE, "attn_prefill.h"), os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, ptxas_verbose: bool = False, jobs: int | None = None) -> str:
    """Compile every kernel translation unit and link the library; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(OUT, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        return obj, r.stderr

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=jobs or min(8, len(srcs))) as ex:
        binding = ex.submit(compile_binding, nvcc)
        results = list(ex.map(compile_one, srcs))
        binding.result()
    if ptxas_verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    link_binding()
    return LIB


def _torch() -> str:
    """PyTorch's folder, found without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch not found: its headers are required to build the binding")
    return spec.submodule_search_locations[0]


def _run(what: str, cmd: list) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stderr}")


def compile_binding(nvcc: str) -> None:
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    torch = os.path.join(_torch(), "include")
    _run("g++ failed on binding.cpp",
         [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-isystem", cuda, "-isystem", torch,
          "-isystem", os.path.join(torch, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
          "-c", os.path.join(CSRC, "binding.cpp"), "-o", os.path.join(OUT, "binding.o")])


def link_binding() -> None:
    """The CPython extension next to the library, which it finds by its own folder; PyTorch's
    own libraries are there by the time it is loaded."""
    tmp = BINDING + f".tmp{os.getpid()}"
    _run("the binding does not link",
         [shutil.which("g++") or "c++", "-shared", "-o", tmp, os.path.join(OUT, "binding.o"), "-L", OUT,
          "-l:" + os.path.basename(LIB), "-L", os.path.join(_torch(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
          "-lc10_cuda", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, BINDING)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv))
