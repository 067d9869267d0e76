"""Build libattnprefill.so in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` compiles to an object in parallel, then nvcc links the
shared library (CUDA runtime linked statically). Then g++ builds the small CPython
extension that marshals the serving-step calls to it, where PyTorch is installed: C
hosts need the library alone. Run as a module
(``python -m chunked_prefill_gqa_gb300.build``) or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libattnprefill.so")
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
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        [os.path.join(INCLUDE, "attn_prefill.h"), os.path.abspath(__file__)]


def binding_path() -> str | None:
    """The binding for this Python and the installed PyTorch, whose tensors it reads in
    place: a layout that another build of either need not share, so both are in its
    name. None without PyTorch."""
    torch = _torch()
    if torch is None:
        return None
    with open(os.path.join(torch, "version.py")) as f:
        got = dict(re.findall(r"^(__version__|git_version)\s*(?::[^=]*)?=\s*['\"]([^'\"]+)", f.read(), re.M))
    tag = "-".join([sysconfig.get_config_var("SOABI"), "torch", got["__version__"], got.get("git_version", "")[:8]])
    return os.path.join(OUT, f"_binding.{tag}.so")


def _binding_deps():
    return [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "attn_prefill.h"), os.path.abspath(__file__)]


def _newer(path: str, deps: list) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and (_torch() is None or _newer(binding_path(), _binding_deps()))


def build(force: bool = False, ptxas_verbose: bool = False, jobs: int | None = None) -> str:
    """Compile every kernel translation unit and link the library; returns its path."""
    os.makedirs(OUT, exist_ok=True)
    library, torch = force or not _newer(LIB, _deps()), _torch()
    binding = torch is not None and (force or not _newer(binding_path(), _binding_deps()))
    with cf.ThreadPoolExecutor(max_workers=1) as ex:  # beside the library, which it must not keep from being linked
        compiled = ex.submit(compile_binding, torch) if binding else None
        if library:
            build_library(ptxas_verbose, jobs)
        if compiled:
            compiled.result()
            link_binding(torch)
    if library and torch is None:
        sys.stderr.write("PyTorch is not installed: the binding of the serving-step calls is not built\n")
    return LIB


def build_library(ptxas_verbose: bool = False, jobs: int | None = None) -> None:
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
        results = list(ex.map(compile_one, srcs))
    if ptxas_verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def _torch() -> str | None:
    """PyTorch's folder, found without importing it; None where it is not installed."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def _run(what: str, cmd: list) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stderr}")


def compile_binding(torch: str) -> None:
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    include = os.path.join(torch, "include")
    _run("g++ failed on binding.cpp",
         [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-isystem", cuda, "-isystem", include,
          "-isystem", os.path.join(include, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
          "-c", os.path.join(CSRC, "binding.cpp"), "-o", os.path.join(OUT, "binding.o")])


def link_binding(torch: str) -> None:
    """The CPython extension next to the library, which it finds by its own folder; PyTorch's
    own libraries are there by the time it is loaded."""
    path = binding_path()
    tmp = path + f".tmp{os.getpid()}"
    _run("the binding does not link",
         [shutil.which("g++") or "c++", "-shared", "-o", tmp, os.path.join(OUT, "binding.o"), "-L", OUT,
          "-l:" + os.path.basename(LIB), "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
          "-lc10_cuda", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, path)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv))
