"""A mixture-of-experts layer for generation steps: experts in NVFP4, a few tokens at a time; and the tokens'
way to the experts of a training batch and back (gather_tokens, combine_tokens over moe_sort's order).

"Nemotron NVFP4" explainer, "The model underneath" (expert layers) and "The honest part: this is
not end-to-end FP4" (the expert weights are what runs in NVFP4). The layer holds the weights, the
routing rule and the workspace that nvfp4_moe_tokens needs; every arithmetic step is in the library's
kernels.
"""
from __future__ import annotations

import torch

from . import (MoESort, MoEWeights, NVFP4Error, NVFP4Tensor, _moe_call, _on_stream, moe_combine, moe_combine_grad, moe_gather,
               moe_workspace, quantize)
from .first_order import first_order


class MoETokens:
    """y = sum over a token's top_k experts of weight * w2 act(w1 x), for up to max_tokens tokens.

    router [experts, hidden] (bfloat16 or float32); w1 [experts*ffn, hidden] (gated: [experts*2*ffn,
    hidden], each expert's gate rows before its up rows) and w2 [experts*hidden, ffn] as NVFP4 tensors
    with one global scale per expert. The layer keeps the tensors it is made with. Calls share one
    workspace: on different streams, order them.
    """

    def __init__(self, router: torch.Tensor, w1: NVFP4Tensor, w2: NVFP4Tensor, top_k: int, activation: str = "relu2",
                 gated: bool = False, score: str = "softmax", renormalize: bool = True, routed_scale: float = 1.0,
                 max_tokens: int = 64):
        self.weights = MoEWeights(router, w1, w2, top_k, activation, gated, score, renormalize, routed_scale)
        self.max_tokens = max_tokens
        self.workspace = moe_workspace(self.weights, max_tokens)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()        # the first call may be on any stream, and needs the zeros
        self._layer = self.weights.c()                       # checked once; addresses of:
        self._kept = (router, *(t for w in (w1, w2) for t in (w.codes, w.scales, w.global_scale)))

    @classmethod
    def from_bf16(cls, router: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, top_k: int, **kw):
        """From weights w1 [experts, ffn (2 ffn), hidden] and w2 [experts, hidden, ffn], quantized in
        16x16 blocks with one tensor scale per expert, as the training layers quantize them."""
        return cls(router, *(_expert_stack(w) for w in (w1, w2)), top_k, **kw)

    @_on_stream
    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, ids_out: torch.Tensor | None = None,
                 weights_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        if x.dim() != 2 or x.shape[0] > self.max_tokens:
            raise NVFP4Error(f"x must be [tokens, hidden] with at most {self.max_tokens} tokens")
        return _moe_call(x, self._layer, out, ids_out, weights_out, self.workspace, stream)


def _expert_stack(w: torch.Tensor) -> NVFP4Tensor:
    if w.dim() != 3 or not w.is_contiguous():
        raise NVFP4Error("expert weights must be a contiguous [experts, rows, cols] tensor")
    experts, rows, cols = w.shape
    segments = torch.arange(experts + 1, dtype=torch.int64, device=w.device) * rows
    return quantize(w.reshape(experts * rows, cols), "16x16", "rn", segments=segments)[0]


class _GatherFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, sort):
        ctx.sort, ctx.dtype = sort, x.dtype
        return moe_gather(x.contiguous(), sort)

    @staticmethod
    @first_order
    def backward(ctx, dxs):
        if dxs.dtype not in (torch.bfloat16, torch.float32):
            dxs = dxs.float()
        return moe_combine(dxs.contiguous(), ctx.sort, out_dtype=ctx.dtype), None


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, sort, out_dtype):
        y, w = y.contiguous(), weights.contiguous()
        ctx.sort = sort
        ctx.save_for_backward(y, w)
        return moe_combine(y, sort, w, out_dtype=out_dtype)

    @staticmethod
    @first_order
    def backward(ctx, dout):
        y, w = ctx.saved_tensors
        # dy leaves the kernel in dout's type: of FP32 rows in FP32, for a pass over dout, which has the fewest rows
        if dout.dtype not in (torch.bfloat16, torch.float32) or y.dtype == torch.float32:
            dout = dout.float()
        dy, dw = moe_combine_grad(dout.contiguous(), y, ctx.sort, w, need_dy=ctx.needs_input_grad[0],
                                  need_dweights=ctx.needs_input_grad[1])
        return None if dy is None else dy.to(y.dtype), dw, None, None


def gather_tokens(x: torch.Tensor, sort: MoESort) -> torch.Tensor:
    """x [tokens, hidden] (bfloat16 or float32) in the order of the experts [sort.rows, hidden], zeros in the rows
    without a pair, with autograd (moe_gather; backward moe_combine)."""
    return _GatherFn.apply(x, sort)


def combine_tokens(y: torch.Tensor, sort: MoESort, weights: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The experts' outputs y [sort.rows, hidden] back in the tokens' order, weighted (weights float32 [tokens,
    top_k]) and added up, with autograd for y and weights (moe_combine; backward moe_combine_grad)."""
    return _CombineFn.apply(y, weights, sort, out_dtype)
