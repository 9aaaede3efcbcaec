"""A stack of SwiGLU MLP blocks: y_l = block_l(y_{l-1}), trained end to end.

Forward keeps, per layer, only what the block's backward needs beyond its
weights: the layer input x_l (which is the previous layer's output, already
kept) and preact_l -- the drop-h saved-tensor policy applied to every layer
("SwiGLU MLP Drop-H technical report", 4-layer stack memory table).  Backward
walks the layers in reverse; each layer's dx is the next (lower) layer's dy.
Every product runs in the library's kernels through the C ABI.  With dropout, y_l =
dropout(block_l(y_{l-1})) in place, and the backward computes each layer's mask again.  Every buffer is the
stack's own, so both directions can be captured into a graph.
"""
from __future__ import annotations

import torch

from . import binding


class SwiGLUStack:
    def __init__(self, layers, M: int, device=None, dropout: float = 0.0, seed: int | None = None):
        """layers: list of (W1 [2H,D], W2 [Dout,H]) CUDA bf16 tensors with D == Dout.  dropout:
        probability of dropping an element of a layer's output; the masks follow from seed, the number of the
        forward call (``calls`` so far, which a resumed run sets, and ``seed``) or forward's step, and the
        layer.  Without a seed the stack draws one of its own with torch's default generator."""
        if not 0 <= dropout <= 1:
            raise ValueError(f"dropout: {dropout}, expected 0 .. 1")
        if dropout and seed is None:
            seed = binding.draw_seed()
        self.dropout, self.seed, self.calls = dropout, seed, 0
        self._masks = None
        self.layers = layers
        self.M = M
        W1, W2 = layers[0]
        self.D = W1.shape[1]
        self.H = W2.shape[1]
        self.Dout = W2.shape[0]
        if self.D != self.Dout:
            raise ValueError("a stack needs D == Dout")
        self.dev = W1.device if device is None else torch.device(device)
        bf = dict(dtype=torch.bfloat16, device=self.dev)
        L = len(layers)
        self.acts = [torch.empty(M, self.D, **bf) for _ in range(L + 1)]     # x_0 .. x_L (= y)
        self.preacts = [torch.empty(M, 2 * self.H, **bf) for _ in range(L)]
        self.grads = [(torch.empty(2 * self.H, self.D, **bf), torch.empty(self.Dout, self.H, **bf)) for _ in range(L)]
        self.dacts = [torch.empty(M, self.D, **bf) for _ in range(2)]        # ping-pong dy / dx
        self.ws_f = torch.empty(max(16, binding.swiglu_mlp_fwd_workspace_size(M, self.D, self.H, self.Dout)),
                                dtype=torch.uint8, device=self.dev)
        self.ws_b = torch.empty(max(16, binding.swiglu_mlp_bwd_workspace_size(M, self.D, self.H, self.Dout)),
                                dtype=torch.uint8, device=self.dev)

    def forward(self, x, step=None):
        """step: an int64 scalar on the device, 0 .. 2**47 - 1, that takes the place of the number of the call in
        the masks.  A captured graph has to have one, and its user to advance it from replay to replay; it is
        left alone between a forward and its backward."""
        self._masks = self._masks_of(step) if self.dropout else None
        self._check_capture()
        self.acts[0].copy_(x)
        self.calls += 1
        for l, (W1, W2) in enumerate(self.layers):
            binding.swiglu_mlp_fwd(self.acts[l], W1, W2, self.preacts[l], self.acts[l + 1], self.ws_f)
            if self._masks:
                binding.swiglu_mlp_dropout(self.acts[l + 1], y=self.acts[l + 1], **self._masks[l])
        return self.acts[-1]

    def _masks_of(self, step):
        """The dropout's arguments for each layer.  With a step the masks are far from those of any call's number."""
        if self.seed is None:      # dropout set since
            self.seed = binding.draw_seed()
        L = len(self.layers)
        offsets = [(self.calls + 1) * L + l if step is None else (l << 48) + (1 << 47) for l in range(L)]
        return [dict(p=self.dropout, seed=self.seed, offset=o, step=step) for o in offsets]

    def _check_capture(self):
        """The number of the call would be a constant of a captured graph."""
        if self._masks and self._masks[0]["step"] is None and torch.cuda.is_current_stream_capturing():
            raise ValueError("step: a captured forward with dropout needs one, or every replay drops the same elements")

    def backward(self, dy):
        """Returns (dx of the stack input, [(dW1_l, dW2_l) for each layer])."""
        self._check_capture()
        cur = dy
        for l in range(len(self.layers) - 1, -1, -1):
            W1, W2 = self.layers[l]
            dW1, dW2 = self.grads[l]
            out = self.dacts[l % 2]
            if self._masks:        # the caller's dy stays as it is
                cur = binding.swiglu_mlp_dropout(cur, y=self.dacts[(l + 1) % 2] if cur is dy else cur, **self._masks[l])
            binding.swiglu_mlp_bwd(self.acts[l], W1, W2, self.preacts[l], cur, out, dW1, dW2, self.ws_b)
            cur = out
        return cur, self.grads

    def saved_activation_bytes(self) -> int:
        """What the forward keeps for the backward beyond the weights: every layer's
        input (x_0 .. x_{L-1}), every preact, and the output."""
        t = self.acts + self.preacts
        return sum(a.numel() * a.element_size() for a in t)

    def backward_peak_bytes(self) -> int:
        """Device memory held at the backward's peak beyond the weights, x and dy (the
        caller's): the saved activations, the backward workspace (h and grad_preact of
        one layer), the dx ping-pong buffers and every layer's weight gradients.  The
        forward's workspace (h) is idle during the backward and not counted."""
        extra = [self.ws_b] + self.dacts + [g for pair in self.grads for g in pair]
        return self.saved_activation_bytes() + sum(a.numel() * a.element_size() for a in extra)
