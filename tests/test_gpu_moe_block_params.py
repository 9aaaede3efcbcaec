"""GPU test of the pre-norm MoE block over torch.nn.Parameters, which a model's weights usually are."""
import pytest
import torch

from helpers import ensure_library

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def test_parameters_train_as_tensors_do():
    ensure_library()
    from bwd_gemm_epilogue_gb300.moe_block import PreNormMoE
    g = torch.Generator().manual_seed(3)
    T, E, D, H, k = 300, 6, 128, 64, 2
    shapes = ((D,), (D,), (E, D), (E, 2 * H, D), (E, D, H))
    weights = [(torch.randn(s, generator=g) * s[-1] ** -0.5).to(bf).cuda() for s in shapes]
    x, dy = (torch.randn(T, D, generator=g).to(bf).cuda() for _ in range(2))

    def train(params):
        block = PreNormMoE(*params, top_k=k)
        out = []
        for _ in range(2):
            y, dx = block.forward(x), block.backward(dy)
            assert not y.requires_grad and not dx.requires_grad, "the block has a backward of its own"
            out += [y, dx, block.step(lr=0.05, max_norm=1.0)]
        return out + block.params + [block.decode(x[:9])]

    want = train([w.clone() for w in weights])
    got = train([torch.nn.Parameter(w.clone()) for w in weights])
    assert all(torch.equal(p, q) for p, q in zip(got, want))
