"""GB300-native SwiGLU MLP block: forward, and a backward whose activation-gradient
GEMM grad_h = dy @ W2 carries the SwiGLU backward in its epilogue; also the residual
block, a mixture-of-experts layer of such blocks, an FP8 forward, layer norm, gradient
clipping, a routed mixture-of-experts layer for a few tokens, and tokens on their way to
experts and back (gate, sort, dispatch, combine) and dropout, with their gradients.

The compute path is a C-ABI shared library of hand-written sm_103a kernels
(``csrc/``, declared in ``include/swiglu_mlp.h``, ``include/swiglu_moe.h``,
``include/swiglu_ops.h`` and ``include/swiglu_tokens.h``); ``binding`` marshals arguments to it with ctypes.  Importing this package does not
load the library; the first call into ``binding`` does, and raises if it has not
been built.  ``stack`` (stacked blocks), ``pipeline`` (steps on host batches) and
``moe_block`` (a pre-norm mixture-of-experts block) sit on top of ``binding``.
"""
__all__ = ["binding", "workloads", "ledger", "stack", "pipeline", "moe_block"]
