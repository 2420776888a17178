"""A linear layer whose three GEMMs run in NVFP4 on the library's kernels (autograd wrapper).

artiverse.ca "NVIDIA's 4-bit floating point pushes AI training limits" (paragraph on which
parts run in 4-bit) and the "Nemotron NVFP4" explainer ("Why 4-bit training normally falls
apart - and the three fixes") give the recipe this wrapper strings together; every step is a
call into libnvfp4, the wrapper only orders the calls and holds the buffers:

  forward   X [T, in] (BF16)  -> 1x16, nearest           -> Xq
            W [out, in]       -> 16x16, nearest, + W^T   -> Wq, WqT
            Y = Xq Wq^T, stored in BF16, with max|Y| from the GEMM epilogue (so the next
            layer's input quantization is a single pass: pass it as ``x_amax``)
  backward  dY [T, out]       -> max|dY| and max|H dY| from one read (amax pair); BF16 or
            FP32 gradients are quantized as they are
            dY -> 1x16, stochastic rounding                   -> dYq
            dX = dYq WqT^T, stored in BF16
            dY, X -> 16-point random-sign Hadamard transform along tokens, then 1x16 along
            tokens (dY stochastic, X nearest)                 -> (H dY)^T, (H X)^T
            dW = (H dY)^T (H X)^T^T in FP32, added into ``main_grad`` (or returned in the
            weight's dtype when the layer keeps no FP32 main gradient)

With a bias, an activation or a residual the forward's last step is one call (gemm_act): Y =
act(Xq Wq^T + b) + R in BF16, with max|Y| and, for the backward, the pre-activation in BF16; the
backward then begins with act_grad: dZ = dY act'(Z) in BF16 (also of an FP32 dY: it goes to 4 bits
next, and Z, whose slope it is, has no more), the bias gradient (added into ``bias_main_grad``
like the weight's) and, for the residual, dY itself.

With checkpoint="fp8" the input X and the pre-activation wait for the backward pass in 8 bits (fp8_quantize: 1.03
bytes per element instead of 2); the weight gradient's operand is then H X of the 8-bit X (rht_quantize of it), the
activation's slope that of the 8-bit pre-activation (act_grad of it). The forward pass does not change.

Stochastic rounding draws from Philox4x32-10 keyed by the layer's seed; call n of the layer's
backward uses counter offsets 2n (activation gradient) and 2n + 1 (weight gradient), so every
call draws fresh bits and a run is reproducible. Tokens (T) must be a multiple of 16 (the
Hadamard block), and in/out features multiples of 16 (the quantization block).
"""
from __future__ import annotations

import torch

from . import (ACTIVATIONS, FP8Tensor, NVFP4Error, _check_q, act_grad, amax, amax_pair, fp8_quantize, gemm_act, gemm_ex, quantize,
               rht_quantize)
from .first_order import first_order


def _state_of(weight):
    """Differs after torch has changed or replaced the weight's values."""
    return weight.data_ptr(), 0 if weight.is_inference() else weight._version


def _save(ctx, layer, t, z, x_fp8):
    """Keeps the input t, if the weight's gradient is wanted, and the pre-activation z (or None) for the backward pass."""
    ctx.eight = layer.checkpoint == "fp8"
    ctx.tokens = t.shape[0]
    if not ctx.needs_input_grad[1]:
        t = None
    if not ctx.eight:
        ctx.save_for_backward(t, z)
        return
    kept = [None if t is None else fp8_quantize(t) if x_fp8 is None else x_fp8, None if z is None else fp8_quantize(z)]
    ctx.eight_shapes = [None if e is None else (e.rows, e.cols) for e in kept]
    ctx.save_for_backward(*(a for e in kept if e is not None for a in (e.codes, e.scales)))


def _saved(ctx):
    """The input and the pre-activation as _save kept them: tensors, or FP8Tensors, or None."""
    if not ctx.eight:
        return ctx.saved_tensors
    buffers = iter(ctx.saved_tensors)
    return [None if shape is None else FP8Tensor(next(buffers), next(buffers), *shape) for shape in ctx.eight_shapes]


def _check_fp8(x_fp8, t, layer):
    if x_fp8 is not None:
        if layer.checkpoint != "fp8":
            raise NVFP4Error('x_fp8 is of use to a layer with checkpoint="fp8"')
        if (x_fp8.rows, x_fp8.cols) != tuple(t.shape):
            raise NVFP4Error(f"x_fp8 shape ({x_fp8.rows}, {x_fp8.cols}) is not x's, {tuple(t.shape)}")
        _check_q(x_fp8, what="x_fp8")
        if not x_fp8.codes.device == x_fp8.scales.device == t.device:
            raise NVFP4Error(f"x_fp8 is not on x's device, {t.device}")


class _LinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, layer, x_amax, x_fp8, train):
        t = x.reshape(-1, x.shape[-1])
        if t.dtype != torch.bfloat16:
            raise NVFP4Error("the NVFP4 linear layer takes BF16 activations")
        t = t.contiguous()
        if t.shape[0] % 16:
            raise NVFP4Error(f"tokens ({t.shape[0]}) must be a multiple of 16")
        _check_fp8(x_fp8, t, layer)
        hx_amax = None                                       # taken in backward
        if x_amax is None:
            if layer.checkpoint == "bf16":
                pair = amax_pair(t, layer.sign_mask)         # max|X|, max|H X| from one read
                x_amax, hx_amax = pair[0:1], pair[1:2]
            else:                                            # the backward's X is the 8-bit one
                x_amax = amax(t)
        qx, _ = quantize(t, "1x16", "rn", amax=x_amax)
        qw, qwt = quantize(weight, "16x16", "rn", amax=layer.weight_amax, emit_transposed=True)
        y_amax = torch.empty((1,), dtype=torch.float32, device=t.device)
        y = gemm_ex(qx, qw, out_dtype=torch.bfloat16, amax_out=y_amax)
        layer.last_output_amax = y_amax
        ctx.layer = layer
        ctx.call = layer._calls
        layer._calls += 1
        ctx.hx_amax = hx_amax
        ctx.x_shape = x.shape
        ctx.weight_dtype = weight.dtype
        if train:
            _save(ctx, layer, t, None, x_fp8)
        ctx.qwt = qwt
        return y.view(*x.shape[:-1], weight.shape[0])

    @staticmethod
    @first_order
    def backward(ctx, dy):
        t, _ = _saved(ctx)
        if ctx.tokens == 0:
            return dy.new_zeros(ctx.x_shape), _nothing(ctx, 1, ctx.layer.weight, ctx.layer.main_grad), None, None, None, None
        g = dy.reshape(-1, dy.shape[-1])
        if g.dtype not in (torch.bfloat16, torch.float32):
            g = g.float()                                    # exact widening; FP32 goes in as is
        dx, dw = _gradient_gemms(ctx, t, g.contiguous())
        return dx.view(ctx.x_shape), dw, None, None, None, None


def _nothing(ctx, i, param, main_grad):
    """The gradient of input i, a parameter, from a call without tokens (an expert that got none)."""
    return torch.zeros_like(param) if ctx.needs_input_grad[i] and main_grad is None else None


def _gradient_gemms(ctx, t, g):
    """dX and dW (None when it went into main_grad, or the weight is frozen) of one call from its input
    t (for dW alone) and the gradient g of its product."""
    layer = ctx.layer
    pair = amax_pair(g, layer.sign_mask)                     # max|dY|, max|H dY| from one read
    qdy, _ = quantize(g, "1x16", "sr", seed=layer.seed, offset=2 * ctx.call, amax=pair[0:1])
    dx = gemm_ex(qdy, ctx.qwt, out_dtype=torch.bfloat16)
    if not ctx.needs_input_grad[1]:
        return dx, None
    hx_amax = ctx.hx_amax
    if hx_amax is None and not isinstance(t, FP8Tensor):     # (of an 8-bit input rht_quantize takes it)
        hx_amax = amax(t, rht=True, sign_mask=layer.sign_mask)
    qhdy = rht_quantize(g, layer.sign_mask, "sr", seed=layer.seed, offset=2 * ctx.call + 1,
                        amax=pair[1:2])
    qhx = rht_quantize(t, layer.sign_mask, "rn", amax=hx_amax)
    dw = None
    if layer.main_grad is not None:
        gemm_ex(qhdy, qhx, out=layer.main_grad, accumulate=True)
    else:
        out_dtype = ctx.weight_dtype if ctx.weight_dtype in (torch.bfloat16, torch.float32) else torch.float32
        dw = gemm_ex(qhdy, qhx, out_dtype=out_dtype).to(ctx.weight_dtype)   # rounded in the epilogue
    return dx, dw


class _LinearActFn(torch.autograd.Function):
    """The same with bias, activation and residual in the forward GEMM's epilogue."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, layer, x_amax, x_fp8, train):
        t = x.reshape(-1, x.shape[-1])
        if t.dtype != torch.bfloat16:
            raise NVFP4Error("the NVFP4 linear layer takes BF16 activations")
        t = t.contiguous()
        if train and t.shape[0] % 16:
            raise NVFP4Error(f"tokens ({t.shape[0]}) must be a multiple of 16")
        _check_fp8(x_fp8, t, layer)
        hx_amax = None
        if x_amax is None:
            if train and layer.checkpoint == "bf16":
                pair = amax_pair(t, layer.sign_mask)
                x_amax, hx_amax = pair[0:1], pair[1:2]
            else:
                x_amax = amax(t)
        qx, _ = quantize(t, "1x16", "rn", amax=x_amax)
        if layer.frozen is not None and not train:
            if layer._frozen_of != _state_of(weight):
                layer.freeze()
            qw, qwt = layer.frozen, None
        else:
            qw, qwt = quantize(weight, "16x16", "rn", amax=layer.weight_amax, emit_transposed=train)
        r = None
        if residual is not None:
            if residual.shape != (*x.shape[:-1], weight.shape[0]):
                raise NVFP4Error(f"residual shape {tuple(residual.shape)} is not the output's")
            r = residual.reshape(-1, weight.shape[0]).contiguous()
        z = (torch.empty((t.shape[0], weight.shape[0]), dtype=torch.bfloat16, device=t.device)
             if train and layer.activation != "none" else None)
        y_amax = torch.empty((1,), dtype=torch.float32, device=t.device)
        y = gemm_act(qx, qw, bias=bias, activation=layer.activation, residual=r, preact=z, amax_out=y_amax)
        layer.last_output_amax = y_amax
        ctx.layer, ctx.hx_amax, ctx.x_shape, ctx.weight_dtype, ctx.qwt = layer, hx_amax, x.shape, weight.dtype, qwt
        if train:
            ctx.call = layer._calls
            layer._calls += 1
            _save(ctx, layer, t, z, x_fp8)
        return y.view(*x.shape[:-1], weight.shape[0])

    @staticmethod
    @first_order
    def backward(ctx, dy):
        layer = ctx.layer
        t, z = _saved(ctx)
        dr = dy if ctx.needs_input_grad[3] else None
        if ctx.tokens == 0:
            return (dy.new_zeros(ctx.x_shape), _nothing(ctx, 1, layer.weight, layer.main_grad),
                    _nothing(ctx, 2, layer.bias, layer.bias_main_grad), dr, None, None, None, None)
        g = dy.reshape(-1, dy.shape[-1])
        if g.dtype not in (torch.bfloat16, torch.float32):
            g = g.float()
        g = g.contiguous()
        db = None
        if ctx.needs_input_grad[2]:
            db = layer.bias_main_grad
            if db is None:
                db = torch.empty((g.shape[1],), dtype=torch.float32, device=g.device)
        dz = g
        if z is not None or db is not None:
            out = act_grad(g, z, activation=layer.activation, dbias=db,
                           accumulate=layer.bias_main_grad is not None, bias_only=z is None)
            dz = g if z is None else out
        dx, dw = _gradient_gemms(ctx, t, dz)
        if layer.bias_main_grad is not None:
            db = None
        elif db is not None:
            db = db.to(layer.bias.dtype)
        return dx.view(ctx.x_shape), dw, db, dr, None, None, None, None


class NVFP4Linear(torch.nn.Module):
    """y = activation(x W^T + bias) + residual with NVFP4 GEMMs; W is a BF16 parameter [out, in].

    bias, activation: none by default; the bias is an FP32 parameter [out], the activation one of
    "none", "relu2", "gelu", "silu"; the residual is an argument of the call.
    main_grad: with ``fp32_main_grad`` (default) the weight gradient is accumulated into the
    FP32 tensor ``self.main_grad`` (zero it between optimizer steps) and ``weight.grad`` stays
    None; otherwise ``weight.grad`` receives it in BF16. ``bias_main_grad`` and ``bias.grad``
    (FP32) likewise. A weight or bias with requires_grad False gets no gradient.
    checkpoint: "bf16", or "fp8": how the input and the pre-activation are kept for the backward pass; with "fp8" an
    input that is there in 8 bits already (RMSNorm's last_output_fp8) can be passed as ``x_fp8``.
    last_output_amax: max|y| of the latest forward (a device float [1]), the ``x_amax`` of a
    following NVFP4Linear.
    weight_amax: None, or a device float [1] holding max|W| (optim.AdamW sets it at every step), which
    makes the weight's quantization a single pass. It holds for the weight as it is when this is set:
    once torch has changed or replaced the weight (load_state_dict, an in-place operation) it reads
    None. torch counts no writes through ``weight.data``, to a weight made in inference mode, or by
    other libraries: after those set it to None (and freeze() again).
    """

    def __init__(self, in_features: int, out_features: int, device=None, sign_mask: int = 0x6E04,
                 seed: int = 0, fp32_main_grad: bool = True, bias: bool = False, activation: str = "none",
                 checkpoint: str = "bf16"):
        super().__init__()
        if in_features % 16 or out_features % 16:
            raise NVFP4Error("in_features and out_features must be multiples of 16")
        if activation not in ACTIVATIONS:
            raise NVFP4Error(f"unknown activation {activation!r}: one of {', '.join(ACTIVATIONS)}")
        if checkpoint not in ("bf16", "fp8"):
            raise NVFP4Error(f"unknown checkpoint {checkpoint!r}: bf16 or fp8")
        self.weight = torch.nn.Parameter(torch.empty((out_features, in_features), dtype=torch.bfloat16,
                                                     device=device))
        self.main_grad = (torch.zeros((out_features, in_features), dtype=torch.float32, device=device)
                          if fp32_main_grad else None)
        self.bias = (torch.nn.Parameter(torch.zeros((out_features,), dtype=torch.float32, device=device))
                     if bias else None)
        self.bias_main_grad = (torch.zeros((out_features,), dtype=torch.float32, device=device)
                               if bias and fp32_main_grad else None)
        self.activation, self.checkpoint = activation, checkpoint
        self.sign_mask = sign_mask & 0xFFFF
        self.seed = seed
        self._calls = 0
        self.last_output_amax = None
        self.weight_amax = None
        self.frozen = self._frozen_of = None

    @property
    def weight_amax(self):
        value, of = self._weight_amax
        return value if of == _state_of(self.weight) else None

    @weight_amax.setter
    def weight_amax(self, value):
        self._weight_amax = value, _state_of(self.weight)

    def forward(self, x: torch.Tensor, x_amax: torch.Tensor | None = None,
                residual: torch.Tensor | None = None, x_fp8: FP8Tensor | None = None) -> torch.Tensor:
        # autograd hides the grad mode from a Function's forward
        train = torch.is_grad_enabled() and any(
            a is not None and a.requires_grad for a in (x, self.weight, self.bias, residual))
        if self.bias is None and self.activation == "none" and residual is None and self.frozen is None:
            return _LinearFn.apply(x, self.weight, self, x_amax, x_fp8, train)
        return _LinearActFn.apply(x, self.weight, self.bias, residual, self, x_amax, x_fp8, train)

    def freeze(self):
        """Quantizes the weight once for the calls without gradients that follow (generation: any
        number of tokens, down to one). A call that finds the weight changed (an optimizer's step,
        load_state_dict: what weight_amax sees) quantizes it anew."""
        with torch.no_grad():
            self.frozen, _ = quantize(self.weight, "16x16", "rn", amax=self.weight_amax)
        self._frozen_of = _state_of(self.weight)
        return self

    def unfreeze(self):
        self.frozen = None
        return self
