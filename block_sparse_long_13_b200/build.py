"""Build libmsa.so (the MSA C-ABI library) in-tree for sm_100a with nvcc, and _bind.so (the Python calls that are made
for every token, natively) with g++ against the installed torch.  Only the first is needed: without the second, Python
makes the same calls by itself.

    python -m block_sparse_long_13_b200.build [--force]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmsa.so")
BIND = os.path.join(HERE, "_bind.so")
BIND_MADE_FOR = os.path.join(HERE, "_bind.made_for")     # the torch and Python that _bind.so was compiled against
ROOT = os.path.dirname(HERE)
HEADER = os.path.join(ROOT, "include", "msa.h")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "-use_fast_math",
    "-Xcompiler", "-fPIC", "-shared",
]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def sources():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh"))] + [HEADER]


def bind_sources():
    return [os.path.join(CSRC, "bind.cpp"), HEADER]


def up_to_date(lib: str = LIB, made_of=None) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(s) <= t for s in (sources() if made_of is None else made_of))


def bind_versions() -> str:
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}, cxx11 abi {int(torch.compiled_with_cxx11_abi())}"


def bind_fits() -> bool:
    """Whether _bind.so is there and was compiled against the torch and Python that run."""
    try:
        with open(BIND_MADE_FOR) as f:
            return os.path.exists(BIND) and f.read() == bind_versions()
    except OSError:
        return False


def _run(cmd, lib: str, verbose: bool) -> None:
    tmp = lib + ".tmp"
    cmd = [*cmd, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)


def build_bind(verbose: bool = False) -> None:
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    if os.path.exists(BIND_MADE_FOR):
        os.remove(BIND_MADE_FOR)
    includes = [sysconfig.get_paths()["include"], os.path.join(at, "include"),
                os.path.join(at, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *[x for i in includes for x in ("-isystem", i)],
          os.path.join(CSRC, "bind.cpp"), "-L" + os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
          "-ltorch_python"], BIND, verbose)
    with open(BIND_MADE_FOR + ".tmp", "w") as f:
        f.write(bind_versions())
    os.replace(BIND_MADE_FOR + ".tmp", BIND_MADE_FOR)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not up_to_date():
        _run([nvcc_path(), *NVCC_FLAGS, os.path.join(CSRC, "msa.cu")], LIB, verbose)
    if force or not bind_fits() or not up_to_date(BIND, bind_sources()):
        try:
            build_bind(verbose)
        except (OSError, subprocess.CalledProcessError) as e:
            print(f"_bind.so was not built ({e}); the calls over the 8-bit cache go through ctypes, which costs some "
                  "microseconds a call", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
