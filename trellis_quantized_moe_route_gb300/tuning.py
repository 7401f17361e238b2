"""Autograd forms of the router losses and of the route combine.

What tuning the router of a layer with frozen experts needs: the gradient goes
from the layer's output through ``combine`` to the route weights, and with the
losses' own through ``route`` to the logits. The experts' rows are constants
here (``binding.MxFp4Experts`` has no backward pass); ``combine`` does return
their gradient to a caller whose rows want one.
"""
from __future__ import annotations

import torch

from . import binding


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, mask):
        r = binding.router_forward(logits, k, mask=mask)
        ctx.save_for_backward(logits, mask, *r)
        ctx.mark_non_differentiable(r.ids, r.lse, r.counts, r.prob, r.tokens)
        return tuple(r)

    @staticmethod
    def backward(ctx, _ids, grad_w, _lse, _counts, _prob, grad_losses, _tokens):
        logits, mask, *r = ctx.saved_tensors
        grad_w = None if grad_w is None else grad_w.contiguous()
        grad_losses = None if grad_losses is None else grad_losses.contiguous()
        return binding.router_backward(logits, binding.RouterOut(*r), grad_w, grad_losses, mask=mask), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, w):
        ctx.save_for_backward(rows, w)
        return binding.combine(rows, w)

    @staticmethod
    def backward(ctx, grad_out):
        rows, w = ctx.saved_tensors
        want_rows, want_w = ctx.needs_input_grad
        return binding.combine_backward(rows, w, grad_out.contiguous(), want_rows, want_w)


def route(logits, k: int, mask=None) -> binding.RouterOut:
    """binding.router_forward with a gradient through ``w`` and ``losses``."""
    return binding.RouterOut(*_Route.apply(logits, k, mask))


def combine(rows, w):
    """binding.combine with a gradient through ``rows`` and ``w``."""
    return _Combine.apply(rows, w)
