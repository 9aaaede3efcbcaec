"""A rule of the sources of moe_gate.cu and moe_tokens.cu that no run on a GPU can show (CPU only): their
launches come up before the kernel ahead of them in the stream has ended, so each kernel waits for it
before it touches memory.  What one without the wait reads depends on timing."""
import os
import re

from test_ops_rules import SOURCES, kernels


def test_every_kernel_that_comes_up_early_waits_first():
    checked = 0
    for path in SOURCES:
        source = open(path).read()
        if "launch_early" not in source:
            continue
        for name, body in kernels(path):
            wait = body.find("after_previous();", 1)
            assert wait >= 0, name
            before = re.sub(r"constexpr [^;]*;|(extern )?__shared__ [^;]*;", "", body[1:wait])
            assert not before.strip(), f"{name}: {before.strip()} comes before the wait"
            checked += 1
    assert checked >= 10


def test_only_these_sources_launch_early():
    assert {os.path.basename(p) for p in SOURCES if "launch_early" in open(p).read()} == {"moe_gate.cu", "moe_tokens.cu"}
