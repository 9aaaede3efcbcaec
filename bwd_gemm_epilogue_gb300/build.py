"""Compile the CUDA library (``libswiglu_mlp.so``) in-tree for sm_103a with nvcc.

One translation unit per file of ``csrc/*.cu`` and ``csrc/ops/*.cu``, compiled in parallel and linked
into one shared library with the CUDA runtime linked statically; beside it a Python module
(``_short_calls.so``, from ``csrc/ops/short_calls.cpp`` with g++ and torch's headers) that makes the
usual calls of the short operators.  Rebuilds only when a source or header is newer than the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libswiglu_mlp.so")
MODULE = os.path.join(HERE, "_short_calls.so")
OBJDIR = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build the library")
    return exe


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MODULE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MODULE))
    deps = glob.glob(os.path.join(CSRC, "*.*")) + glob.glob(os.path.join(CSRC, "ops", "*.*")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _compile_module(cuda_home: str) -> str:
    """The object of the Python module, against the torch that imports it."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(OBJDIR, "short_calls.o")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    f"-I{INCLUDE}", f"-I{inc}", f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
                    f"-I{os.path.join(cuda_home, 'include')}", f"-I{sysconfig.get_paths()['include']}", "-c",
                    os.path.join(CSRC, "ops", "short_calls.cpp"), "-o", obj], check=True)
    return obj


def _link_module(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MODULE + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:" + os.path.basename(LIB), f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
                    "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(tmp, MODULE)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    nvcc = _nvcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "ops", "*.cu")))

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        module = ex.submit(_compile_module, os.path.dirname(os.path.dirname(os.path.realpath(nvcc))))
        objs = list(ex.map(compile_one, srcs))
        module_obj = module.result()
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static"], check=True)
    os.replace(tmp, LIB)
    _link_module(module_obj)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
