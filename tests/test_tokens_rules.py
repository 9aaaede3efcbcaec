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


def test_what_a_warp_does_together_stands_in_no_short_circuit():
    """Shuffles, votes and reductions name every lane of the warp, so none may be the second operand of ||,
    && or ?:, which some lanes would not reach."""
    together = r"(?:Group<G>::(?:max|sum|of)|__shfl\w*|__any_sync|__all_sync|__ballot_sync|__reduce_\w+|__match_\w+|warp_sums?)\("
    for path in SOURCES:
        if os.path.basename(path) not in ("moe_gate.cu", "moe_tokens.cu"):
            continue
        for i, line in enumerate(open(path).read().split("\n"), 1):
            code = line.split("//")[0]
            assert not re.search(rf"(?:\|\||&&|\?)[^;)]*{together}", code), f"{os.path.basename(path)}:{i}: {code.strip()}"
