"""The root-mean-square norm in front of a layer, with the residual stream's addition (autograd wrapper).

artiverse.ca "NVIDIA's 4-bit floating point pushes AI training limits" (paragraph on which parts run in
4-bit): norms and the residual stream stay in higher precision. The arithmetic is nvfp4_rms_norm's and
nvfp4_rms_norm_grad's; the wrapper orders the calls and holds the buffers.
"""
from __future__ import annotations

import torch

from . import FP8Tensor, NVFP4Error, rms_norm, rms_norm_grad
from .first_order import first_order


class _NormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, layer):
        t = x.reshape(-1, x.shape[-1]).contiguous()
        r = None
        if residual is not None:
            if residual.shape != x.shape or residual.dtype != x.dtype:
                raise NVFP4Error(f"residual {tuple(residual.shape)} {residual.dtype} is not like x, {tuple(x.shape)} {x.dtype}")
            r = residual.reshape(t.shape).contiguous()
        h = torch.empty_like(t) if r is not None else None
        q = FP8Tensor.empty(*t.shape, device=t.device) if layer.fp8 else None
        amax = torch.empty((1,), dtype=torch.float32, device=t.device)
        y = rms_norm(t, weight, residual=r, eps=layer.eps, residual_out=h, fp8_out=q, amax_out=amax)
        layer.last_output_amax, layer.last_output_fp8 = amax, q
        ctx.set_materialize_grads(False)                     # an output without a gradient costs none
        ctx.save_for_backward(t if h is None else h, weight)
        ctx.eps, ctx.shape, ctx.two = layer.eps, x.shape, h is not None
        return y.view(x.shape) if h is None else (y.view(x.shape), h.view(x.shape))

    @staticmethod
    @first_order
    def backward(ctx, dy, dh=None):
        h, weight = ctx.saved_tensors
        dr = None if dh is None else dh.reshape(h.shape).to(h.dtype).contiguous()
        dw = None
        if dy is None:
            dx = dr
        else:
            g = dy.reshape(h.shape)
            if g.dtype not in (torch.bfloat16, torch.float32):
                g = g.float()
            if ctx.needs_input_grad[2]:
                dw = torch.empty(weight.shape, dtype=torch.float32, device=h.device)
            dx = rms_norm_grad(g.contiguous(), h, weight, dresidual=dr, eps=ctx.eps, dweight=dw)
        if dx is not None:
            dx = dx.view(ctx.shape)
        return dx, dx if ctx.two else None, None if dw is None else dw.to(weight.dtype), None


class RMSNorm(torch.nn.Module):
    """y = h / sqrt(mean(h^2) + eps) * weight in BF16 over the last dimension, h = x, or x + residual.

    forward(x) returns y; forward(x, residual) returns (y, h), h being the residual stream to go on with, in
    x's dtype (bfloat16 or float32). weight: float32 [features], ones at first.
    last_output_amax: max|y| of the latest forward (a device float [1]), the ``x_amax`` of a following NVFP4Linear.
    fp8: the latest y is also left in 8 bits in last_output_fp8 (an FP8Tensor), the ``x_fp8`` of a following
    NVFP4Linear with 8-bit checkpoints.
    """

    def __init__(self, features: int, eps: float = 1e-6, device=None, fp8: bool = False):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones((features,), dtype=torch.float32, device=device))
        self.eps, self.fp8 = eps, fp8
        self.last_output_amax = self.last_output_fp8 = None

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        return _NormFn.apply(x, residual, self.weight, self)
