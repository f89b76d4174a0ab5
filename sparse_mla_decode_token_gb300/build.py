"""Build the C-ABI shared library ``_build/libsmla.so`` for sm_103a, and the
extension module ``_build/smla_torch.so`` that calls it with torch tensors.

Every ``csrc/*.cu`` translation unit is compiled by nvcc in parallel with one
``-gencode arch=compute_103a,code=sm_103a`` target, then linked into one shared
library; ``csrc/cache_torch.cpp`` (host code) is compiled beside them.  Set ``SMLA_PTXAS_VERBOSE=1`` to print register / shared-memory use.
"""
from __future__ import annotations

import concurrent.futures as cf
import fcntl
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libsmla.so")
TORCH_SRC = os.path.join(CSRC, "cache_torch.cpp")
TORCH_EXT = os.path.join(BUILD, "smla_torch.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = GENCODE + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                        "-Xcompiler", "-Wall", "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the library needs the CUDA toolkit to build")
    return path


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "smla.h"))
    return files


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def _run(what: str, cmd: list[str]) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_torch_ext() -> str:
    import torch
    home = os.path.dirname(os.path.dirname(nvcc()))
    root = os.path.dirname(torch.__file__)
    obj = TORCH_SRC[:-4].replace(CSRC, BUILD) + ".o"
    _run("g++", ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                 "-I", INCLUDE, "-isystem", os.path.join(root, "include"),
                 "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                 "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(home, "include"),
                 "-c", TORCH_SRC, "-o", obj])
    return obj


def _link_torch_ext(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = TORCH_EXT + ".tmp"
    _run("link", ["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-lsmla", "-Wl,-rpath,$ORIGIN", "-L", libs, "-lc10",
                  "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, TORCH_EXT)


def build(force: bool = False, verbose: bool | None = None) -> str:
    """Compile (if stale) and return the path of ``libsmla.so``."""
    if verbose is None:
        verbose = os.environ.get("SMLA_PTXAS_VERBOSE", "0") == "1"
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, "lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)              # processes that find it stale together build it once
        if not force and not verbose and not _stale(LIB, _deps()) and not _stale(TORCH_EXT, _deps()):
            return LIB
        srcs = sources()
        with cf.ThreadPoolExecutor(max_workers=max(2, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
            ext = ex.submit(_compile_torch_ext)
            objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
            ext_obj = ext.result()
        tmp = LIB + ".tmp"
        _run("link", [nvcc()] + GENCODE + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB)
        _link_torch_ext(ext_obj)
        return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv or None))
