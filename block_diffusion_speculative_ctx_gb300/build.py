"""Build the dflash shared library in-tree with nvcc for sm_103a.

Each .cu file is compiled to an object in parallel, then linked into
``_build/libdflash.so``.  No CMake; only nvcc and the CUDA runtime.  Beside it, where torch's
headers are installed, the host compiler makes the Python operators' argument checks
(``csrc/tensor_args.cpp``, a CPython extension); without it ops.py checks in Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(BUILD, "libdflash.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the dflash CUDA library cannot be built")


def sources() -> list:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(f) for f in files) if files else 0.0


def up_to_date() -> bool:
    return os.path.exists(LIB) and os.path.getmtime(LIB) >= max(_deps_mtime(), os.path.getmtime(__file__))


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def tensor_args_path():
    """Where the argument-check extension for this interpreter and this torch lies (built or not); None
    without torch."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return None
    with open(os.path.join(torch_dir, "version.py"), "rb") as f:
        tag = hashlib.sha1(f.read() + torch_dir.encode() + sys.version.encode()).hexdigest()[:12]
    return os.path.join(BUILD, f"_tensor_args_{tag}.so")


def _build_tensor_args(path: str):
    torch_dir, src = _torch_dir(), os.path.join(CSRC, "tensor_args.cpp")
    if os.path.exists(path) and os.path.getmtime(path) >= os.path.getmtime(src):
        return
    tmp = path + f".{os.getpid()}.tmp"
    lib = os.path.join(torch_dir, "lib")
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", "-I" + os.path.join(torch_dir, "include"),
           "-I" + os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), "-I" + sysconfig.get_paths()["include"],
           "-I" + os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), src, "-o", tmp, "-L" + lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath," + lib]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        print(f"argument checks stay in Python: {e}", file=sys.stderr)
        return
    if r.returncode != 0:
        print(f"argument checks stay in Python: {r.stderr[-2000:]}", file=sys.stderr)
        return
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    path = tensor_args_path()
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        checks = ex.submit(_build_tensor_args, path) if path else None
        lib = _build_lib(force, verbose, extra_flags)
        if checks:
            checks.result()
    return lib


def _build_lib(force: bool, verbose: bool, extra_flags) -> str:
    if not force and up_to_date():
        return LIB
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
