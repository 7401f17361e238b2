"""Autograd forms of the router losses, the route combine, the products by
expert, the distillation loss and the token log probabilities.

What tuning the router of a layer with frozen experts needs: the gradient goes
from the layer's output through ``combine`` to the route weights, and with the
losses' own through ``route`` to the logits. Frozen experts' rows are constants
(``binding.MxFp4Experts`` has no backward pass); experts in 16 bits take part
through ``experts``, which has the gradients of its rows and weights. ``distill``
and ``token_logprobs`` are the losses at the head. Gradients are of first order:
a second derivative through any of them is refused.
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
        raise RuntimeError("route, combine, experts, distill and token_logprobs have first-order gradients only")


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


class _Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, plan, per_route):
        ctx.save_for_backward(x, w)
        ctx.plan, ctx.per_route = plan, per_route
        return binding.experts_forward(x, w, plan, per_route=per_route)

    @staticmethod
    def backward(ctx, grad_out):
        x, w = ctx.saved_tensors
        want_x, want_w = ctx.needs_input_grad[:2]
        grad_out = grad_out.contiguous()
        grad_x, grad_w = binding.experts_backward(x, w, ctx.plan, grad_out, ctx.per_route, want_x, want_w)
        return _first_order(grad_x, w, grad_out), _first_order(grad_w, x, grad_out), None, None


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, values, temperature, mask, teacher_lse):
        r = binding.distill_forward(logits, ids, values, temperature, mask, teacher_lse)
        ctx.save_for_backward(logits, ids, values, mask, teacher_lse, r.stats)
        ctx.temperature = temperature
        return r.loss

    @staticmethod
    def backward(ctx, grad_loss):
        logits, ids, values, mask, teacher_lse, stats = ctx.saved_tensors
        grad_loss = grad_loss.contiguous()
        grad = binding.distill_backward(logits, ids, values, binding.DistillOut(None, stats), grad_loss, ctx.temperature,
                                        mask, teacher_lse)
        return _first_order(grad, logits, grad_loss), None, None, None, None, None


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, top, temperature):
        r = binding.token_logprobs(logits, targets, top, temperature)
        ctx.save_for_backward(logits, targets, r.entropy, r.stats)
        ctx.temperature = temperature
        ctx.mark_non_differentiable(r.top_ids, r.top_logprobs, r.stats)
        ctx.set_materialize_grads(False)  # (a loss of the log probabilities alone: no entropy term)
        return tuple(r)

    @staticmethod
    def backward(ctx, grad_logprob, grad_entropy, _ids, _logprobs, _stats):
        if grad_logprob is None and grad_entropy is None:
            return None, None, None, None
        logits, targets, entropy, stats = ctx.saved_tensors
        grad_logprob = None if grad_logprob is None else grad_logprob.contiguous()
        grad_entropy = None if grad_entropy is None else grad_entropy.contiguous()
        fwd = binding.TokenLogprobs(None, entropy, None, None, stats)
        grad = binding.token_logprobs_backward(logits, targets, fwd, grad_logprob, grad_entropy, ctx.temperature)
        return _first_order(grad, logits, grad_logprob, grad_entropy), None, None, None


def experts(x, w, plan: binding.ExpertPlan, per_route: bool = False):
    """binding.experts_forward with a gradient through ``x`` and ``w``. Whether the
    products and gradients are right is in the plan's error word: a training loop asks
    ``plan.poll_error()``, which waits for the stream, after its backward pass."""
    return _Experts.apply(x, w, plan, per_route)


def distill(logits, ids, values, temperature: float = 1.0, mask=None, teacher_lse=None):
    """The losses [T] of binding.distill_forward with a gradient through
    ``logits``; the teacher is a constant."""
    for name, t in (("values", values), ("teacher_lse", teacher_lse)):
        if t is not None and t.requires_grad:
            raise ValueError("%s requires a gradient: the teacher is a constant of the loss" % name)
    return _Distill.apply(logits, ids, values, temperature, mask, teacher_lse)


def token_logprobs(logits, targets, top: int = 0, temperature: float = 1.0) -> binding.TokenLogprobs:
    """binding.token_logprobs with a gradient through ``logprob`` and ``entropy``."""
    return binding.TokenLogprobs(*_TokenLogprobs.apply(logits, targets, top, temperature))
