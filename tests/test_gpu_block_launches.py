"""GPU test of what the pre-norm MoE block has torch do beside its own kernels."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from test_gpu_moe_block import batch, params
from test_gpu_tokens import b  # noqa: F401

pytestmark = pytest.mark.gpu


class Conversions(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.types = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten._to_copy.default and out.is_cuda:
            self.types.append(out.dtype)
        return out


def test_a_training_step_converts_rows_and_router_only(b):  # noqa: F811
    """xn and a bf16 router to fp32 for their products, in each direction, and the router's gradient back."""
    from bwd_gemm_epilogue_gb300.moe_block import PreNormMoE
    block = PreNormMoE(*params(4, 64, 32, 1, torch.bfloat16), top_k=2)
    x, dy = batch(40, 64, 2), batch(40, 64, 3)
    with Conversions() as seen:
        block.forward(x)
        block.backward(dy)
    assert seen.types == [torch.float32] * 4 + [torch.bfloat16]
