"""Compile the CUDA library (``libswiglu_mlp.so``) in-tree for sm_103a with nvcc.

One translation unit per file of ``csrc/*.cu`` and ``csrc/ops/*.cu``, compiled in parallel and linked
into one shared library with the CUDA runtime linked statically.  Beside it a Python module
(``_short_calls.so``, from ``csrc/ops/short_calls.cpp`` with g++ and torch's headers) that makes the
usual calls of the short operators in less host time; where it does not build (no torch, no Python or
torch headers) there is a warning, and the library, which needs none of them, stands without it.
Each is rebuilt only when one of its sources or headers is newer, the module also when the torch or
the Python that imports it is another.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libswiglu_mlp.so")
MODULE = os.path.join(HERE, "_short_calls.so")
MODULE_SOURCE = os.path.join(CSRC, "ops", "short_calls.cpp")
OBJDIR = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build the library")
    return exe


def _newer(deps, target: str) -> bool:
    """Whether the target is missing, or older than one of deps."""
    return not os.path.exists(target) or any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def _stale_library() -> bool:
    deps = [os.path.join(CSRC, "*.*"), os.path.join(CSRC, "ops", "*.cu*"), os.path.join(INCLUDE, "*.h")]
    return _newer([f for d in deps for f in glob.glob(d)], LIB)


def _module_key() -> str:
    """What the module is built against: a torch that has CUDA, and this Python."""
    import torch
    if torch.version.cuda is None:
        raise ImportError("this torch was built without CUDA")
    return f"{torch.__version__} {os.path.dirname(torch.__file__)} {sysconfig.get_config_var('SOABI')}"


def _key_path() -> str:
    return os.path.join(OBJDIR, "short_calls.key")


def _stale_module() -> bool:
    if _newer([MODULE_SOURCE, *glob.glob(os.path.join(INCLUDE, "*.h"))], MODULE) or not os.path.exists(_key_path()):
        return True
    with open(_key_path()) as f:
        return f.read() != _module_key()


def _compile_module(cuda_home: str) -> str:
    """The object of the Python module, against the torch that imports it."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(OBJDIR, "short_calls.o")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    f'-DSWIGLU_TORCH="{torch.__version__}"', f"-I{INCLUDE}", f"-I{inc}",
                    f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}", f"-I{os.path.join(cuda_home, 'include')}",
                    f"-I{sysconfig.get_paths()['include']}", "-c", MODULE_SOURCE, "-o", obj], check=True)
    return obj


def _link_module(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MODULE + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{os.path.dirname(LIB)}", "-l:" + os.path.basename(LIB), f"-L{lib}",
                    "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(tmp, MODULE)
    with open(_key_path(), "w") as f:
        f.write(_module_key())


def _build_library(nvcc: str, verbose: bool) -> None:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "ops", "*.cu")))

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static"], check=True)
    os.replace(tmp, LIB)


def _module_object(force: bool):
    """The module's object, or None where the module is up to date."""
    if not force and not _stale_module():
        return None
    return _compile_module(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))))


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(_module_object, force)              # beside the library's own units
        if force or _stale_library():
            _build_library(_nvcc(), verbose)
    try:
        obj = module.result()
        if obj is not None:
            _link_module(obj)
    except (ImportError, OSError, RuntimeError, subprocess.CalledProcessError) as e:
        if os.path.exists(MODULE):                             # of other sources, or for another torch
            os.remove(MODULE)
        warnings.warn(f"{os.path.basename(MODULE)} was not built ({e}); the short operators' calls go through ctypes")
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
