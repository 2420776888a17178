"""First derivatives only: what the package's backward passes return cannot be differentiated again.

The kernels behind them are no torch operations, so under create_graph=True their results would be constants to autograd,
and a penalty on a gradient would add nothing to the gradients of a loss without a word. With this around a Function's backward it
raises where it is differentiated; gradients that are kept as a graph but not differentiated stay what they are.
"""
from __future__ import annotations

import functools

import torch

from . import NVFP4Error


class _End(torch.autograd.Function):
    @staticmethod
    def forward(ctx, grad):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise NVFP4Error("there is no second derivative: the gradients of this package's layers cannot be differentiated")


def first_order(backward):
    @functools.wraps(backward)
    def ending(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        # (a gradient that is passed on as it came keeps its own graph)
        return tuple(g if g is None or any(g is given for given in grads) else _End.apply(g.detach().requires_grad_()) for g in out)
    return ending
