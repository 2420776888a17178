"""A language model's output head and its loss, without the logits (autograd wrapper).

artiverse.ca "NVIDIA's 4-bit floating point pushes AI training limits" (paragraph on which parts run in
4-bit): the output head stays in BF16. The arithmetic is nvfp4_linear_cross_entropy's and its gradient's.
"""
from __future__ import annotations

import torch

from . import NVFP4Error, linear_cross_entropy, linear_cross_entropy_grad
from .first_order import first_order


class _HeadFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, layer, train):
        t = x.reshape(-1, x.shape[-1]).contiguous()
        loss, lse = linear_cross_entropy(t, weight, targets)
        if train:                                            # a copy: the caller may change the loss that it gets
            ctx.save_for_backward(t, weight, targets, lse, loss.clone())
        ctx.layer, ctx.x_shape = layer, x.shape
        return loss

    @staticmethod
    @first_order
    def backward(ctx, grad):
        t, weight, targets, lse, loss = ctx.saved_tensors
        main = ctx.layer.main_grad
        dx, dw = linear_cross_entropy_grad(t, weight, targets, lse, grad.float().contiguous(), dweight=main, accumulate=main is not None,
                                           need_dx=ctx.needs_input_grad[0], need_dweight=ctx.needs_input_grad[1], loss=loss)
        return None if dx is None else dx.view(ctx.x_shape), None if main is not None else dw, None, None, None


class LinearCrossEntropy(torch.nn.Module):
    """Cross entropy of softmax(x weight^T) with the targets; weight is a BF16 parameter [vocab, hidden].

    forward(x [..., hidden] BF16, targets [...] int64): a target outside 0 .. vocab - 1 (as -100) does not
    count. reduction: "mean" over the targets that count (0 if none does), "sum", or "none" (float32, the targets' shape).
    main_grad: with ``fp32_main_grad`` (default) the weight gradient is accumulated into the FP32 tensor
    ``self.main_grad``, as NVFP4Linear's, and ``weight.grad`` stays None; otherwise ``weight.grad`` receives it in BF16.
    (Either way its addends are of softmax gradients held in BF16, the targets' in twice as many bits.)
    """

    bias = bias_main_grad = None                             # as NVFP4Linear without a bias

    def __init__(self, hidden: int, vocab: int, device=None, reduction: str = "mean", fp32_main_grad: bool = True):
        super().__init__()
        if hidden % 16:
            raise NVFP4Error("hidden must be a multiple of 16")
        if reduction not in ("mean", "sum", "none"):
            raise NVFP4Error(f"unknown reduction {reduction!r}: mean, sum or none")
        self.weight = torch.nn.Parameter(torch.empty((vocab, hidden), dtype=torch.bfloat16, device=device))
        self.main_grad = torch.zeros((vocab, hidden), dtype=torch.float32, device=device) if fp32_main_grad else None
        self.reduction = reduction

    def forward(self, x: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        if targets.shape != x.shape[:-1]:
            raise NVFP4Error(f"targets shape {tuple(targets.shape)} is not x's, {tuple(x.shape[:-1])}")
        flat = targets.reshape(-1).contiguous()
        train = torch.is_grad_enabled() and (x.requires_grad or self.weight.requires_grad)   # hidden from a Function's forward
        loss = _HeadFn.apply(x, self.weight, flat, self, train)
        if self.reduction == "none":
            return loss.view(targets.shape)
        if self.reduction == "sum":
            return loss.sum()
        return loss.sum() / ((flat >= 0) & (flat < self.weight.shape[0])).sum().clamp_min(1)
