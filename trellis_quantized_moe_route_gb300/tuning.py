"""Autograd forms of the router losses and of the route combine.

What tuning the router of a layer with frozen experts needs: the gradient goes
from the layer's output through ``combine`` to the route weights, and with the
losses' own through ``route`` to the logits. The experts' rows are constants
here (``binding.MxFp4Experts`` has no backward pass); ``combine`` does return
their gradient to a caller whose rows want one. Gradients are of first order: a
second derivative through either is refused.
"""
from __future__ import annotations

import torch

from . import binding


class _FirstOrder(torch.autograd.Function):
    """A gradient as it is, that refuses to be differentiated in turn."""

    @staticmethod
    def forward(ctx, grad, *sources):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("route and combine have first-order gradients only")


def _first_order(grad, *sources):
    """`grad`, made by a kernel from `sources`. Where a graph of the backward
    pass is being built (create_graph) it depends on all of them, though no
    operation shows it: also where the incoming gradient is a constant, which is
    all that once_differentiable looks at."""
    if grad is not None and torch.is_grad_enabled() and any(s is not None and s.requires_grad for s in sources):
        return _FirstOrder.apply(grad, *sources)
    return grad


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
        grad = binding.router_backward(logits, binding.RouterOut(*r), grad_w, grad_losses, mask=mask)
        return _first_order(grad, logits, grad_w, grad_losses), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, w):
        ctx.save_for_backward(rows, w)
        return binding.combine(rows, w)

    @staticmethod
    def backward(ctx, grad_out):
        rows, w = ctx.saved_tensors
        want_rows, want_w = ctx.needs_input_grad
        grad_out = grad_out.contiguous()
        grad_rows, grad_w = binding.combine_backward(rows, w, grad_out, want_rows, want_w)
        return _first_order(grad_rows, w, grad_out), _first_order(grad_w, rows, grad_out)


def route(logits, k: int, mask=None) -> binding.RouterOut:
    """binding.router_forward with a gradient through ``w`` and ``losses``."""
    return binding.RouterOut(*_Route.apply(logits, k, mask))


def combine(rows, w):
    """binding.combine with a gradient through ``rows`` and ``w``."""
    return _Combine.apply(rows, w)
