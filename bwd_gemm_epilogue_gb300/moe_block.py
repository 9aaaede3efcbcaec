"""A pre-norm mixture-of-experts block, trained and then served:

    y = x + sum_j gate_j * expert_{e_j}(LayerNorm(x)),   gates = softmax over the top_k logits

``forward`` / ``backward`` / ``step`` train it on batches: layer norm forward and backward with
the residual stream's gradient fused in, the grouped experts (``swiglu_moe_fwd`` / ``_bwd``) on
rows sorted by expert, and gradients clipped by their global norm before the update.  The
routing between them (a [T, E] product, a sort, gathers) is plain torch, and the grouped
launches take their row counts from the host.  ``decode`` answers for up to 64 tokens with the
same weights in a handful of launches and no host synchronisation (``swiglu_moe_routed_fwd``).
"""
from __future__ import annotations

import torch

from . import binding


class PreNormMoE:
    """gamma, beta [D], router [E, D] (fp32 or bf16), W1 [E, 2H, D], W2 [E, D, H] bf16 CUDA tensors or
    Parameters; the block has a backward of its own, and autograd sees nothing of it."""

    def __init__(self, gamma, beta, router, W1, W2, top_k: int, eps: float = 1e-5):
        E, H2, D = W1.shape
        if W2.shape != (E, D, H2 // 2) or router.shape != (E, D) or gamma.shape != (D,) or beta.shape != (D,):
            raise ValueError(f"shape mismatch: gamma {tuple(gamma.shape)}, beta {tuple(beta.shape)}, router "
                             f"{tuple(router.shape)}, W1 {tuple(W1.shape)}, W2 {tuple(W2.shape)}")
        if not 1 <= top_k <= E:
            raise ValueError(f"top_k: {top_k}, expected 1 .. {E}")
        self.params = [gamma, beta, router, W1, W2]
        self.top_k, self.eps = top_k, eps
        self.grads = None
        self._saved = None

    @torch.no_grad()
    def forward(self, x):
        """x [T, D] bf16 -> y [T, D]; keeps what the backward needs."""
        gamma, beta, router, W1, W2 = self.params
        T, k = x.shape[0], self.top_k
        xn, _, mean, rstd = binding.swiglu_mlp_layer_norm_fwd(x, gamma, beta, self.eps)
        logits = xn.float() @ router.float().T
        picked, ids = (v[:, :k] for v in torch.sort(logits, dim=1, descending=True, stable=True))
        gates = torch.softmax(picked, dim=1)
        order = torch.argsort(ids.reshape(-1), stable=True)              # (token, choice) pairs by expert
        counts = torch.bincount(ids.reshape(-1), minlength=router.shape[0]).tolist()
        xg = xn[order // k]
        preact, rows = binding.swiglu_moe_fwd(xg, W1, W2, counts)
        out = torch.empty_like(rows)
        out[order] = rows
        out = out.reshape(T, k, -1)
        y = (x.float() + (out.float() * gates[:, :, None]).sum(1)).to(x.dtype)
        self._saved = (x, xn, mean, rstd, ids, gates, order, counts, xg, preact, out)
        return y

    @torch.no_grad()
    def backward(self, dy):
        """dy [T, D] bf16 -> dx; leaves the parameters' gradients in self.grads."""
        gamma, _, router, W1, W2 = self.params
        x, xn, mean, rstd, ids, gates, order, counts, xg, preact, out = self._saved
        T, k = x.shape[0], self.top_k
        dgates = (dy.float()[:, None] * out.float()).sum(2)
        drows = (dy.float()[:, None] * gates[:, :, None]).to(dy.dtype).reshape(T * k, -1)[order]
        dxg, dW1, dW2 = binding.swiglu_moe_bwd(xg, W1, W2, preact, drows, counts)
        back = torch.empty_like(dxg)
        back[order] = dxg
        dpicked = gates * (dgates - (gates * dgates).sum(1, keepdim=True))
        dlogits = torch.zeros(T, router.shape[0], device=x.device).scatter(1, ids, dpicked)
        dxn = back.reshape(T, k, -1).float().sum(1) + dlogits @ router.float()
        drouter = (dlogits.T @ xn.float()).to(router.dtype)
        dx, dgamma, dbeta = binding.swiglu_mlp_layer_norm_bwd(dxn.to(x.dtype), x, gamma, mean, rstd, dskip=dy)
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
