"""Embedding with a scale, as a layer: y = scale * weight[tokens], its gradient summed by sorted
tokens (ops.py; the kernels are in ``libinstant.so``)."""
from __future__ import annotations

import torch

from . import ops


class _EmbeddingFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale, padding):
        ctx.save_for_backward(tokens)
        ctx.vocab, ctx.scale, ctx.padding = weight.shape[0], scale, padding
        return ops.embedding_forward(tokens, weight, scale)

    @staticmethod
    @ops.differentiated_once
    def backward(ctx, gy):
        (tokens,) = ctx.saved_tensors
        return None, ops.embedding_backward(gy.contiguous(), tokens, ctx.vocab, ctx.scale, ctx.padding), None, None


class InstantEmbedding(torch.nn.Module):
    """Rows of weight [V, C] looked up by token (int64 or int32, any shape) and multiplied by scale
    (sqrt(C) in many language models); V <= 2^18, C a multiple of 8, dtype "bf16" or "fp32".

    padding: a token whose row gets no gradient through the lookup (zeros at the start, unless the
    weight is given). weight: where the weight starts. A Parameter of the layer's type and device,
    contiguous, is taken as it is, so it may also be the last product's (tied): hand one Parameter,
    or one layer's weight, to both constructors, and autograd adds the gradients. Anything else is
    copied, and not tied. The gradient is dense [V, C], takes at most 2^22 tokens, has the same bits
    every time, and cannot be differentiated again (create_graph=True raises RuntimeError)."""

    def __init__(self, V, C, scale=1.0, padding=None, dtype="bf16", weight=None, device="cuda"):
        super().__init__()
        if dtype not in ("bf16", "fp32"):
            raise ValueError(f"dtype must be 'bf16' or 'fp32', got {dtype!r}")
        if not 1 <= V <= ops.MAX_VOCAB:
            raise ValueError(f"V must be 1 to {ops.MAX_VOCAB}, got {V}")
        if C < 8 or C % 8:
            raise ValueError(f"C must be a positive multiple of 8, got {C}")
        if padding is not None and not 0 <= padding < V:
            raise ValueError(f"padding must be a token of the vocabulary, got {padding}")
        self.V, self.C, self.scale, self.padding = int(V), int(C), float(scale), padding
        torch_dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        if weight is None:
            weight = torch.randn(self.V, self.C, device=device) * self.C ** -0.5
            if padding is not None:
                weight[padding] = 0
            self.weight = torch.nn.Parameter(weight.to(torch_dtype))
        elif tuple(weight.shape) != (self.V, self.C):
            raise ValueError(f"weight must be [{V}, {C}], got {tuple(weight.shape)}")
        else:
            self.weight = ops.weight_parameter(weight, device, torch_dtype)

    def forward(self, tokens):
        return _EmbeddingFn.apply(tokens.contiguous(), self.weight, self.scale, self.padding)
