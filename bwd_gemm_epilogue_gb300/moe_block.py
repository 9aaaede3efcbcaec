"""A pre-norm mixture-of-experts block, trained and then served:

    y = x + sum_j gate_j * expert_{e_j}(LayerNorm(x)),   gates = softmax over the top_k logits

``forward`` / ``backward`` / ``step`` train it on batches, in the library's kernels but for the
router's two products with torch: layer norm forward and backward with the residual stream's gradient fused
in, the gate (softmax and top k), the rows sorted by expert, the grouped experts
(``swiglu_moe_fwd`` / ``_bwd``) and their rows back to the tokens with the gates, dropout and the
residual stream, each with its gradient, and gradients clipped by their global norm before the
update.  The grouped launches take their row counts from the host, the one synchronisation of a
step.  ``decode`` answers for up to 64 tokens with the same weights in a handful of launches and no
host synchronisation (``swiglu_moe_routed_fwd``).
"""
from __future__ import annotations

import torch

from . import binding


class PreNormMoE:
    """gamma, beta [D], router [E, D] (fp32 or bf16), W1 [E, 2H, D], W2 [E, D, H] bf16 CUDA tensors or
    Parameters; the block has a backward of its own, and autograd sees nothing of it."""

    def __init__(self, gamma, beta, router, W1, W2, top_k: int, eps: float = 1e-5, dropout: float = 0.0,
                 seed: int | None = None, layer: int = 0):
        """dropout: probability of dropping an element of the experts' sum in training (not in
        decode).  The masks follow from seed, layer (0 .. 65535) and the number of the forward call (``calls``
        so far, which a resumed run sets, and ``seed``): the blocks of one model need a seed or a layer each.  Without a
        seed the block draws one of its own with torch's default generator."""
        E, H2, D = W1.shape
        if W2.shape != (E, D, H2 // 2) or router.shape != (E, D) or gamma.shape != (D,) or beta.shape != (D,):
            raise ValueError(f"shape mismatch: gamma {tuple(gamma.shape)}, beta {tuple(beta.shape)}, router "
                             f"{tuple(router.shape)}, W1 {tuple(W1.shape)}, W2 {tuple(W2.shape)}")
        if not 1 <= top_k <= E:
            raise ValueError(f"top_k: {top_k}, expected 1 .. {E}")
        if not 0 <= dropout <= 1:
            raise ValueError(f"dropout: {dropout}, expected 0 .. 1")
        if not 0 <= layer < 1 << 16:
            raise ValueError(f"layer: {layer}, expected 0 .. 65535")
        if dropout and seed is None:
            seed = binding.draw_seed()
        self.params = [gamma, beta, router, W1, W2]
        self.top_k, self.eps = top_k, eps
        self.dropout, self.seed, self.layer, self.calls = dropout, seed, layer, 0
        self.grads = None
        self._kept = None

    @property
    def _saved(self):
        """What the last forward kept, and after rstd its experts in torch's index type, which no kernel needs."""
        return (*self._kept[:4], self._kept[-3].long(), *self._kept[4:])

    @torch.no_grad()
    def forward(self, x):
        """x [T, D] bf16 -> y [T, D]; keeps what the backward needs."""
        gamma, beta, router, W1, W2 = self.params
        xn, _, mean, rstd = binding.swiglu_mlp_layer_norm_fwd(x, gamma, beta, self.eps)
        logits = xn.float() @ router.float().T
        ids, gates = binding.swiglu_moe_gate_fwd(logits, self.top_k)
        counts, pos = binding.swiglu_moe_sort(ids, router.shape[0])
        counts = counts.tolist()
        xg = binding.swiglu_moe_dispatch_fwd(xn, pos, sum(counts))
        preact, rows = binding.swiglu_moe_fwd(xg, W1, W2, counts)
        if self.dropout and self.seed is None:             # dropout set since
            self.seed = binding.draw_seed()
        mask = dict(p=self.dropout, seed=self.seed or 0, offset=(self.layer << 48) + self.calls)
        y = binding.swiglu_moe_combine_fwd(rows, pos, gates, residual=x, **mask)
        self.calls += 1
        self._kept = (x, xn, mean, rstd, gates, logits, counts, xg, preact, rows, ids, pos, mask)
        return y

    @torch.no_grad()
    def backward(self, dy):
        """dy [T, D] bf16 -> dx; leaves the parameters' gradients in self.grads."""
        gamma, _, router, W1, W2 = self.params
        x, xn, mean, rstd, gates, logits, counts, xg, preact, rows, ids, pos, mask = self._kept
        drows, dgates = binding.swiglu_moe_combine_bwd(dy, rows, pos, gates, **mask)
        dxg, dW1, dW2 = binding.swiglu_moe_bwd(xg, W1, W2, preact, drows, counts)
        dlogits = binding.swiglu_moe_gate_bwd(logits, ids, gates, dgates)
        dxn = binding.swiglu_moe_dispatch_bwd(dxg, pos, add=dlogits @ router.float())
        drouter = (dlogits.T @ xn.float()).to(router.dtype)
        dx, dgamma, dbeta = binding.swiglu_mlp_layer_norm_bwd(dxn, x, gamma, mean, rstd, dskip=dy)
        self.grads = [dgamma, dbeta, drouter, dW1, dW2]
        return dx

    @torch.no_grad()
    def step(self, lr: float, max_norm: float):
        """Clip the gradients in place by their global norm and take a plain descent step;
        returns the norm before clipping (on the device)."""
        norm, _ = binding.swiglu_mlp_clip_grads(self.grads, max_norm)
        for p, g in zip(self.params, self.grads):
            p.add_(g, alpha=-lr)
        return norm

    @torch.no_grad()
    def decode(self, x):
        """y of forward for up to 64 tokens, nothing kept."""
        gamma, beta, router, W1, W2 = self.params
        xn = binding.swiglu_mlp_layer_norm_fwd(x, gamma, beta, self.eps)[0]
        return binding.swiglu_moe_routed_fwd(xn, router, W1, W2, self.top_k, residual=x)[0]
