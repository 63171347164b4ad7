"""Build libtfpaged.so in this package directory with nvcc for sm_100a, and
_serve.so, the compiled argument marshalling of serving.py, with g++.

    python -m paged_kv_cache_segment_b200.build [--verbose-ptxas]
    python paged_kv_cache_segment_b200/build.py --lib-only

The second form builds the C library alone, with nvcc and nothing of torch or
Python's headers.  In the first the library is linked before _serve.so, which is
bound to the torch and Python it was built with; _serve.built names them.

The shared library exports exactly the C ABI of include/tfpaged.h and
include/tfserve.h.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtfpaged.so")
EXT = os.path.join(HERE, "_serve.so")
EXT_FOR = os.path.join(HERE, "_serve.built")
EXT_SRC = os.path.join(CSRC, "serve_ext.cpp")
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-shared",
         "--expt-relaxed-constexpr", "-Wno-deprecated-gpu-targets"]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(HERE, "..", "include", "*.h")))


def _older(target: str, files: list[str]) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in files)


def ext_for() -> str:
    """What _serve.so is bound to: this interpreter and torch."""
    import torch

    return f"python {sys.version_info.major}.{sys.version_info.minor} torch {torch.__version__}"


def stale(ext: bool = True) -> bool:
    if _older(LIB, sources() + headers()):
        return True
    if not ext:
        return False
    if _older(EXT, headers() + [EXT_SRC]) or not os.path.exists(EXT_FOR):
        return True
    with open(EXT_FOR) as f:
        return f.read() != ext_for()


def compile_ext(obj: str) -> str:
    """Compile serve_ext.cpp against this interpreter and torch."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ce

    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    inc = [d for p in [*ce.include_paths(), sysconfig.get_paths()["include"], cuda_inc] for d in ("-isystem", p)]
    subprocess.run([CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc, "-c", EXT_SRC, "-o",
                    obj], check=True)
    return obj


def link_ext(obj: str) -> str:
    """Link _serve.so with libtfpaged.so beside it and with torch's libraries (loaded by `import torch`)."""
    import torch

    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    subprocess.run([CXX, "-shared", "-s", obj, "-o", EXT, "-L", HERE, "-l:libtfpaged.so", "-Wl,-rpath,$ORIGIN", "-L",
                    torch_lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"], check=True)
    with open(EXT_FOR, "w") as f:
        f.write(ext_for())
    return EXT


def build(verbose_ptxas: bool = False, force: bool = False, ext: bool = True) -> str:
    """Compile every csrc/*.cu to an object in parallel (one nvcc a file), link
    them into the shared library, then (with `ext`) build _serve.so against it."""
    if not force and not stale(ext):
        return LIB
    from concurrent.futures import ThreadPoolExecutor

    objdir = os.path.join(HERE, "..", "_build")
    os.makedirs(objdir, exist_ok=True)
    inc = ["-I", os.path.join(HERE, "..", "include")]
    compile_flags = [f for f in FLAGS if f != "-shared"]

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [NVCC, *ARCH, *compile_flags, *inc, "-c", src, "-o", obj]
        if verbose_ptxas:
            cmd += ["-Xptxas", "-v"]
        subprocess.run(cmd, check=True)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        ext_obj = ex.submit(compile_ext, os.path.join(objdir, "serve_ext.o")) if ext else None
        objs = list(ex.map(compile_one, sources()))
    subprocess.run([NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", LIB], check=True)
    if ext_obj is not None:
        link_ext(ext_obj.result())
    return LIB


if __name__ == "__main__":
    build(verbose_ptxas="--verbose-ptxas" in sys.argv, force=True, ext="--lib-only" not in sys.argv)
    print(LIB)
