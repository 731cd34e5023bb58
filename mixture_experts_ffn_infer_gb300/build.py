"""Build the CUDA library in-tree: ``mixture_experts_ffn_infer_gb300/libmoe_ffn.so``.

Every translation unit is compiled for sm_103a only (``-gencode
arch=compute_103a,code=sm_103a``), in parallel, then linked into one shared
library with a static CUDA runtime.  The driver API is reached through
``cudaGetDriverEntryPointByVersion``, so loading the library needs no GPU.

Beside it goes ``_mx_torch``, the Python module of the microscaled-format, FP8
and router calls on torch tensors (``csrc/*_torch.cpp``): host code, compiled with g++ against
torch's headers and linked to the library.  Where g++, Python's headers or
torch's are not installed the library is built without it; it is built again
when another torch is installed.

    python -m mixture_experts_ffn_infer_gb300.build [--force] [--verbose]
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_ffn.so")
BINDING = os.path.join(HERE, "_mx_torch" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_SRC = [os.path.join(CSRC, f) for f in ("mx_torch.cpp", "fp8_torch.cpp")]
BINDING_FOR = "mx_torch.for"  # in BUILD: what the module was compiled against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
        os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [os.path.abspath(__file__)]


def _newer(made: str, deps) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(p) <= os.path.getmtime(made) for p in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, sources() + _headers())


def binding_up_to_date() -> bool:
    if not _newer(BINDING, [LIB, *BINDING_SRC] + _headers()):
        return False
    try:
        with open(os.path.join(BUILD, BINDING_FOR)) as f:
            return f.read() == _torch_version()
    except FileNotFoundError:
        return False


def up_to_date() -> bool:
    return library_up_to_date() and (binding_lacks() is not None or binding_up_to_date())


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # not installed as a package: told apart by its place
        return importlib.util.find_spec("torch").origin


def _torch_paths():
    """(include directories, library directory) of the installed torch."""
    root = os.path.dirname(os.path.abspath(importlib.util.find_spec("torch").origin))
    inc = os.path.join(root, "include")
    return [inc, os.path.join(inc, "torch", "csrc", "api", "include")], os.path.join(root, "lib")


def binding_lacks() -> str | None:
    """What the torch module cannot be built without and is not installed here, or None."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    if not os.path.exists(os.path.join(_torch_paths()[0][0], "ATen", "core", "Tensor.h")):
        return "torch's headers"
    if not os.path.exists(os.path.join(_torch_paths()[1], "libc10_cuda.so")):
        return "a torch with CUDA"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    return None if shutil.which("g++") else "g++"


def compile_binding() -> list[str]:
    with cf.ThreadPoolExecutor(max_workers=len(BINDING_SRC)) as ex:
        return list(ex.map(_compile_host, BINDING_SRC))


def _compile_host(src: str) -> str:
    inc, _ = _torch_paths()
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")
    cmd = ["g++", "-std=c++20", "-O2", "-fPIC", "-fvisibility=hidden", "-Wall", "-D_GLIBCXX_USE_CXX11_ABI=1", "-I", INCLUDE, "-I", CSRC,
           *[f"-isystem{p}" for p in (*inc, sysconfig.get_paths()["include"], cuda)], "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def link_binding(objects: list[str]) -> None:
    _, lib = _torch_paths()
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, *objects, "-Wl,--no-as-needed", LIB, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(os.path.join(BUILD, BINDING_FOR), "w") as f:
        f.write(_torch_version())


def build(force: bool = False, verbose: bool = False) -> str:
    lacks = binding_lacks()
    library = force or not library_up_to_date()
    module = lacks is None and (library or not binding_up_to_date())
    if not library and not module:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(compile_binding) if module else None  # the longest: first
        if library:
            build_library(verbose)
        if binding:
            link_binding(binding.result())
        else:
            print(f"built without the calls on torch tensors (mx.py, fp8.py): {lacks} not found", file=sys.stderr)
            if os.path.exists(BINDING):
                os.remove(BINDING)  # of the library before this one
    return LIB


def build_library(verbose: bool = False) -> None:
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, sources()))
    if verbose:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=libmoe_ffn.so", "-o", tmp, *[o for o, _ in results], "-lpthread", "-ldl",
           "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
