"""Log probabilities of given tokens as a layer, with the log of the sum, the entropy and the most
likely alternatives (ops.py; the kernels are in ``libinstant.so``)."""
from __future__ import annotations

import torch

from . import ops


class _TokenLogprobsFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, vocab, top, ignore):
        out = ops.token_logprobs(logits, targets, vocab, top, ignore)
        ctx.save_for_backward(logits, targets, out.stats, out.entropy)
        ctx.vocab, ctx.ignore = vocab, ignore
        ctx.set_materialize_grads(False)
        # (in one call: each replaces the one before)
        ctx.mark_non_differentiable(out.stats, *((out.top_logp, out.top_index) if top else ()))
        return tuple(out)

    @staticmethod
    @ops.differentiated_once
    def backward(ctx, g_logp, g_lse, g_entropy, *_):
        logits, targets, stats, entropy = ctx.saved_tensors
        if g_logp is None and g_lse is None and g_entropy is None:
            return None, None, None, None, None
        g = [None if t is None else t.contiguous() for t in (g_logp, g_lse, g_entropy)]
        gz = ops.token_logprobs_backward(logits, targets, stats, *g, entropy=entropy, vocab=ctx.vocab,
                                         ignore=ctx.ignore)
        return gz, None, None, None, None


def token_logprobs(logits, targets=None, vocab=None, top=0, ignore=ops.IGNORE) -> ops.TokenLogprobs:
    """ops.token_logprobs with gradients: logp, lse and entropy can be differentiated (once:
    create_graph=True raises RuntimeError), the alternatives cannot. A language model's loss is
    -logp.sum() / (targets != ignore).sum(); lse.square() and entropy serve the usual additions to
    it."""
    out = _TokenLogprobsFn.apply(logits.contiguous(), None if targets is None else targets.contiguous(), vocab, top,
                                 ignore)
    return ops.TokenLogprobs(*out)
