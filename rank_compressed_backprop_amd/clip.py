"""Clipping of a model's gradients by their norm (ops.py; the kernels are in ``libinstant.so``)."""
from __future__ import annotations

import torch

from . import ops


def clip_grad_norm_(parameters, max_norm) -> torch.Tensor:
    """Scales the gradients of parameters (one or an iterable) in place so that the norm over all of
    them is at most max_norm, and returns the norm before (float32 on the device; nothing waits for
    it). Parameters without a gradient take no part; one that is listed twice counts once. Gradients
    are contiguous float32 or bfloat16 tensors on the current device."""
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    seen, grads = set(), []
    for p in parameters:
        if p.grad is not None and id(p) not in seen:
            seen.add(id(p))
            grads.append(p.grad)
    if not grads:
        return torch.zeros((), device=parameters[0].device if parameters else None)
    return ops.clip_grads(grads, max_norm)
