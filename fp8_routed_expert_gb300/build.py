"""Build libfp8moe.so (the layer's C ABI and its sm_103a kernels) and
_torch_binding-torch*.so (the native Python binding of the paged attention,
for the Python and torch that run this) in-tree.

Each .cu file is compiled separately and in parallel with nvcc for
compute_103a / sm_103a only, then linked into one shared library next to
this file; the binding is one C++ file against torch's headers.  ``python -m
fp8_routed_expert_gb300.build`` runs it by hand.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

from ._lib import binding_path

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfp8moe.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _compile_binding() -> str:
    """Object file of csrc/torch_binding.cpp."""
    import torch
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "torch_binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", base,
           "-isystem", os.path.join(base, "torch", "csrc", "api", "include"),
           "-c", os.path.join(CSRC, "torch_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed on torch_binding.cpp")
    return obj


def _link_binding(obj: str, path: str) -> None:
    import torch
    tmp = path + f".tmp{os.getpid()}"
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-L", PKG,
           "-l:libfp8moe.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link of the Python binding failed")
    os.replace(tmp, path)


def _build_lib(verbose: bool, extra_flags: list[str]) -> None:
    cc = nvcc()
    flags = NVCC_FLAGS + extra_flags

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cudalib = os.path.join(os.path.dirname(os.path.dirname(cc)), "lib64")
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart", "-L", cudalib,
           "-Xlinker", f"-rpath={cudalib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link of libfp8moe.so failed")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """The C ABI's library, then the Python binding, each where it is missing or
    older than its sources.  The library needs nvcc alone: where the binding
    cannot be built the error says so, and the library is there."""
    def fresh(path: str) -> bool:
        return not force and os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()

    binding = binding_path()
    with_lib, with_binding = not fresh(LIB), not fresh(binding)
    if not (with_lib or with_binding):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_binding) if with_binding else None
        if with_lib:
            _build_lib(verbose, extra_flags or [])
        if obj is not None:
            try:
                _link_binding(obj.result(), binding)
            except Exception as e:
                raise RuntimeError(f"{LIB} is built, the paged attention's Python binding is not: {e}") from e
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
