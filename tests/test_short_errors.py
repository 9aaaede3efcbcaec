"""Errors in the arguments of the compiled calls come out as themselves (CPU only: they are met before
anything reaches a device)."""
import pytest
import torch

from test_ops_checks import b  # noqa: F401


class NoTruth:
    def __bool__(self):
        raise ArithmeticError("neither true nor false")


def test_a_flag_without_a_truth(b):  # noqa: F811
    x, W1, W2 = torch.zeros(3, 8).bfloat16(), torch.zeros(4, 16, 8).bfloat16(), torch.zeros(4, 8, 8).bfloat16()
    with pytest.raises(ArithmeticError, match="neither"):
        b.swiglu_moe_routed_fwd(x, x[:1].expand(4, 8).contiguous(), W1, W2, 2, renormalize=NoTruth())
    with pytest.raises(RuntimeError, match="ambiguous"):
        b.swiglu_moe_routed_fwd(x, x[:1].expand(4, 8).contiguous(), W1, W2, 2, renormalize=torch.ones(2))


def test_numbers_that_are_none(b):  # noqa: F811
    calls = b._short()
    for args in (("one", 0.0), (1.0, None), (1.0, NoTruth())):
        with pytest.raises(TypeError):
            calls.clip_grads([torch.zeros(3)], None, *args)
    with pytest.raises(OverflowError):
        calls.clip_grads([torch.zeros(3)], None, 10 ** 400, 0.0)
