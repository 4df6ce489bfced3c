"""RMS norm with the residual's addition, as a layer: h = x + residual, y = h / rms(h) * weight,
with y also in 8 bits as the next layer's checkpoint (ops.py; the kernels are in
``libinstant.so``)."""
from __future__ import annotations

import torch

from . import ops


class _RMSNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, y8):
        out = ops.rmsnorm_forward(x, weight, residual, eps, y8=y8)
        ctx.save_for_backward(out.h, weight, out.rstd)
        ctx.has_res = residual is not None
        ctx.set_materialize_grads(False)
        q, s = out.y8 if y8 else (None, None)
        if y8:
            ctx.mark_non_differentiable(q, s)
        return out.y, out.h if ctx.has_res else None, q, s

    @staticmethod
    @ops.differentiated_once
    def backward(ctx, gy, gh, *_):
        h, weight, rstd = ctx.saved_tensors
        if gy is None:  # only h was used
            gx, gw = gh, None
        else:
            gx, gw = ops.rmsnorm_backward(gy.contiguous(), h, weight, rstd, None if gh is None else gh.contiguous(),
                                          ctx.needs_input_grad[2])
        return gx, gx if ctx.has_res else None, gw, None, None


class InstantRMSNorm(torch.nn.Module):
    """RMS norm over the last dimension (C channels, a multiple of 8), weight [C] of ones;
    dtype is the type of the weight and of the inputs ("bf16" or "fp32").

    forward(x, residual=None) returns ops.NormOut's y and h: (y, h) with a residual, where
    h = x + residual is the new residual stream, else y. With checkpoint="int8" a Checkpoint8 of
    y follows, for InstantLinear's x8. The gradients cannot be differentiated again (create_graph=True
    raises RuntimeError)."""

    def __init__(self, C, eps=1e-6, dtype="bf16", checkpoint=None, device="cuda"):
        super().__init__()
        if checkpoint not in (None, "int8"):
            raise ValueError(f"checkpoint must be None or 'int8', got {checkpoint!r}")
        if dtype not in ("bf16", "fp32"):
            raise ValueError(f"dtype must be 'bf16' or 'fp32', got {dtype!r}")
        if C < 8 or C % 8:
            raise ValueError(f"C must be a positive multiple of 8, got {C}")
        self.C, self.eps, self.checkpoint = int(C), float(eps), checkpoint
        self.weight = torch.nn.Parameter(torch.ones(self.C, device=device, dtype=torch.bfloat16 if dtype == "bf16"
                                                    else torch.float32))

    def forward(self, x, residual=None):
        y, h, q, s = _RMSNormFn.apply(x.contiguous(), None if residual is None else residual.contiguous(), self.weight,
                                      self.eps, self.checkpoint == "int8")
        out = (y,) if residual is None else (y, h)
        if q is not None:
            out += (ops.Checkpoint8(q, s),)
        return out if len(out) > 1 else y
