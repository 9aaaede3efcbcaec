"""Rules of the operators' sources that no run on a GPU can show (CPU only): what a broken one does
depends on timing."""
import glob
import os
import re

from helpers import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "bwd_gemm_epilogue_gb300", "csrc", "ops", "*.cu")))


def kernels(path):
    """(name, body without comments) of every __global__ function of a source."""
    src = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__global__ .*?(\w+_kernel)\(", src, flags=re.S):
        at = src.index("{", m.end())
        depth, end = 1, at + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
        yield m.group(1), src[at:end]


def test_the_parser_finds_the_kernels():
    names = [n for p in SOURCES for n, _ in kernels(p)]
    assert {"moe_route_kernel", "moe_up_kernel", "grad_squares_kernel", "layer_norm_fwd_kernel"} <= set(names)


def test_shared_memory_of_another_cta_is_touched_only_once_that_cta_runs():
    """Distributed shared memory may be accessed once every CTA of the cluster is known to have
    started, which a wait at the cluster's barrier tells; and a CTA whose memory others access may
    leave only after a second one."""
    checked = 0
    for path in SOURCES:
        for name, body in kernels(path):
            for var in re.findall(r"(\w+) = cluster\.map_shared_rank\(", body):
                access = [m.start() for m in re.finditer(rf"(?<![\w.]){var}\[", body)]
                waits = [m.start() for m in re.finditer(r"cluster\.(?:sync|barrier_wait)\(", body)]
                assert access and waits, name
                assert waits[0] < access[0], f"{name}: {var} accessed before the cluster's barrier"
                assert access[-1] < waits[-1], f"{name}: a CTA may leave while {var} is accessed"
                checked += 1
    assert checked >= 1
