"""The build (CPU only): the C library stands without the Python module, and the calls without it
too."""
import os
import subprocess
import sys
import types

import pytest
import torch

from helpers import ensure_library

CUDA = "must live on a CUDA device"


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """The build with its outputs under tmp_path and its compilers replaced: commands.log has what ran."""
    from bwd_gemm_epilogue_gb300 import build
    for name, path in (("LIB", "libswiglu_mlp.so"), ("MODULE", "_short_calls.so"), ("OBJDIR", "_build")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    log, broken = [], set()

    def run(cmd, check):
        tool = os.path.basename(cmd[0])
        log.append(tool)
        if tool in broken:
            raise subprocess.CalledProcessError(1, cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    return build, log, broken


def test_both_are_built_once(tree):
    build, log, _ = tree
    assert os.path.exists(build.build()) and os.path.exists(build.MODULE)
    assert "nvcc" in log and "g++" in log
    log.clear()
    build.build()
    assert log == []


def test_the_library_is_built_where_the_module_is_not(tree):
    build, log, broken = tree
    broken.add("g++")
    with pytest.warns(UserWarning, match="_short_calls.so was not built"):
        lib = build.build()
    assert os.path.exists(lib) and not os.path.exists(build.MODULE)


def test_without_torch_the_library_is_built(tree, monkeypatch):
    build, log, _ = tree
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(UserWarning, match="_short_calls.so was not built"):
        lib = build.build()
    assert os.path.exists(lib) and not os.path.exists(build.MODULE) and "g++" not in log


def test_another_torch_rebuilds_the_module_alone(tree, monkeypatch):
    build, log, broken = tree
    build.build()
    log.clear()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build()
    assert "g++" in log and "nvcc" not in log
    monkeypatch.setattr(torch, "__version__", "0.0.2")      # and one that it cannot be built for leaves none
    broken.add("g++")
    with pytest.warns(UserWarning, match="_short_calls.so was not built"):
        build.build()
    assert not os.path.exists(build.MODULE)


def test_a_failing_library_still_raises(tree):
    build, _, broken = tree
    broken.add("nvcc")
    with pytest.raises(subprocess.CalledProcessError):
        build.build()


@pytest.mark.parametrize("module", [None, types.SimpleNamespace(torch_version="0.0.1")], ids=["missing", "another torch's"])
def test_calls_without_the_module_go_through_ctypes(monkeypatch, module):
    ensure_library()
    from bwd_gemm_epilogue_gb300 import binding as b
    monkeypatch.setattr(b, "_short_calls", None)
    monkeypatch.setitem(sys.modules, "bwd_gemm_epilogue_gb300._short_calls", module)
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.warns(UserWarning, match="through ctypes"), pytest.raises(ValueError, match=CUDA):
        b.swiglu_mlp_layer_norm_fwd(x)
    with pytest.raises(ValueError, match=CUDA):             # the warning comes once
        b.swiglu_mlp_clip_grads([x], 1.0)


def test_the_module_is_this_torchs():
    ensure_library()
    from bwd_gemm_epilogue_gb300 import binding as b
    assert b._short().torch_version == torch.__version__
