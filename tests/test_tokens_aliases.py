"""Refusals, by the C entry points of include/swiglu_tokens.h, of outputs in an input's place that lie another
way (CPU only: the checks come before anything reaches a device).  Rows of another stride or type are written
over others that have yet to be read."""
import pytest
import torch

from test_ops_checks import A, INVALID, b  # noqa: F401


@pytest.fixture
def refused(b):  # noqa: F811
    """Whether a call is refused for an output's place.  What passes that check fails for want of a device."""
    if torch.cuda.is_available():
        pytest.skip("legal calls with made-up pointers would be launched")

    def check(entry, *args):
        return getattr(b.lib(), entry)(*args, None) == INVALID and b"place" in b.lib().swiglu_mlp_last_error_detail()
    return check


def gate(ld, ldd, renorm, T=4):
    return "swiglu_moe_gate_bwd", A, ld, 2 * A, 3 * A, 4 * A, A, ldd, T, 64, 2, renorm, 0


def dispatch(lda, ldx, type=0, add_type=0, T=4):
    return "swiglu_moe_dispatch_bwd", 2 * A, 64, 3 * A, A, lda, A, ldx, T, 64, 2, 8, type, add_type


def combine(ldr, ldy, T=4):
    return "swiglu_moe_combine_fwd", 2 * A, 64, 3 * A, 4 * A, A, ldr, A, ldy, T, 64, 2, 8, 0, 0.5, 1, 2, None


def dropout(ldx, ldr, ldy, x=A, r=2 * A, M=4):
    return "swiglu_mlp_dropout", x, ldx, r, ldr, A, ldy, M, 64, 0, 0.5, 1, 2, None


def test_rows_of_another_stride(refused):
    assert refused(*gate(64, 72, 0)) and refused(*gate(72, 64, 0))
    assert refused(*dispatch(64, 72)) and refused(*dispatch(72, 64))
    assert refused(*combine(64, 72)) and refused(*combine(72, 64))
    assert refused(*dropout(64, 80, 72)) and refused(*dropout(80, 64, 72, x=2 * A, r=A)) and refused(*dropout(72, 64, 72, r=A))


def test_rows_of_another_type(refused):
    """fp32 to add, a 16-bit gradient."""
    assert refused(*dispatch(64, 64, add_type=2)) and refused(*dispatch(64, 64, 1, 2, T=1))
    assert not refused(*dispatch(64, 64, 2, 2))


def test_what_is_allowed(refused):
    """The same rows; one row, whose stride is nothing; logits that are not read."""
    for call in (gate(72, 72, 0), gate(64, 72, 1), gate(64, 72, 0, T=1), dispatch(72, 72), dispatch(64, 72, T=1), combine(72, 72),
                 combine(64, 72, T=1), dropout(72, 72, 72, r=A), dropout(64, 72, 72, x=2 * A, r=A), dropout(64, 72, 80, M=1, r=A)):
        assert not refused(*call), call
