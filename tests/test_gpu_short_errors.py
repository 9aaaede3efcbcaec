"""GPU tests of errors that the compiled calls pass on from torch."""
import pytest
import torch

from test_gpu_short_calls import BF, b  # noqa: F401

pytestmark = pytest.mark.gpu


def test_no_memory_for_the_outputs_is_torchs_own_error(b):  # noqa: F811
    """What allocates in torch raises torch.OutOfMemoryError, which a caller may catch and answer with
    a smaller batch.  The cap is the allocator's own, on the host."""
    x = torch.ones(1 << 14, 1 << 12, dtype=BF, device="cuda")           # 128 MB, and as much for y
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.empty_cache()
    cap = (torch.cuda.memory_reserved() + (16 << 20)) / total
    torch.cuda.set_per_process_memory_fraction(cap)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            b.swiglu_mlp_layer_norm_fwd(x)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert b.swiglu_mlp_layer_norm_fwd(x)[0].shape == x.shape
