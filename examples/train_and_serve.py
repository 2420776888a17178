"""Trains a small MLP block and a few experts in NVFP4, then serves them one token at a time.

  training  up (bias, squared ReLU) and down (bias, residual) with gemm_act / act_grad and the NVFP4
            gradient GEMMs; the experts likewise, each on the tokens routed to it; one AdamW step for
            all of their tensors, states in 8 bits, gradients clipped
  serving   the block's weights frozen (gemm_act for one row), the experts and their router as one
            expert layer (moe_tokens)

    python examples/train_and_serve.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_block_scaled_quantize_amd.linear import NVFP4Linear  # noqa: E402
from bit_block_scaled_quantize_amd.moe import MoETokens  # noqa: E402
from bit_block_scaled_quantize_amd.optim import AdamW  # noqa: E402

HIDDEN, FFN, EXPERTS, TOKENS = 256, 512, 4, 512


class Mlp(torch.nn.Module):
    def __init__(self, seed, bias):
        super().__init__()
        self.up = NVFP4Linear(HIDDEN, FFN, device="cuda", seed=seed, bias=bias, activation="relu2")
        self.down = NVFP4Linear(FFN, HIDDEN, device="cuda", seed=seed + 1, bias=bias)
        for layer in (self.up, self.down):
            torch.nn.init.normal_(layer.weight, std=layer.weight.shape[1] ** -0.5)

    def forward(self, x, residual=None):
        h = self.up(x)
        return self.down(h, x_amax=self.up.last_output_amax, residual=residual)


class Model(torch.nn.Module):
    """y = mlp(x) + x, then the expert whose router row is nearest (top 1) in its place for half of it."""

    def __init__(self):
        super().__init__()
        self.mlp = Mlp(1, bias=True)
        self.experts = torch.nn.ModuleList(Mlp(10 + 2 * e, bias=False) for e in range(EXPERTS))
        self.register_buffer("router", torch.randn(EXPERTS, HIDDEN, device="cuda").bfloat16())

    def forward(self, x, expert_of):
        y = self.mlp(x, residual=x)
        return y, [self.experts[e](x[expert_of == e]) for e in range(EXPERTS)]


def batch(model, teacher, generator):
    """Tokens in equal numbers near each router row, so that every expert has a multiple of 16."""
    e = torch.arange(TOKENS, device="cuda") % EXPERTS
    x = torch.randn(TOKENS, HIDDEN, device="cuda", generator=generator)
    x = (x + 0.5 * model.router.float()[e]).bfloat16()
    return x, e, x.float() @ teacher, torch.stack([x.float() @ teacher * (0.5 + i) for i in range(EXPERTS)])


def main(steps: int = 60) -> dict:
    torch.manual_seed(0)
    generator = torch.Generator(device="cuda")
    generator.manual_seed(1)
    model = Model()
    teacher = torch.randn(HIDDEN, HIDDEN, device="cuda") * HIDDEN ** -0.5
    opt = AdamW.of(model, lr=2e-3, weight_decay=0.01, states="8bit", max_norm=1.0, seed=7)
    losses = []
    for _ in range(steps):
        x, e, want, want_expert = batch(model, teacher, generator)
        y, parts = model(x, e)
        loss = (y.float() - x.float() - want).square().mean()
        for i, part in enumerate(parts):
            loss = loss + (part.float() - want_expert[i][e == i]).square().mean() / EXPERTS
        loss.backward()
        norm = opt.step()
        opt.zero_grad()
        losses.append(loss.detach())

    # serving: one token through the frozen block, a few through the expert layer
    model.mlp.up.freeze()
    model.mlp.down.freeze()
    layer = MoETokens.from_bf16(model.router, torch.stack([m.up.weight.detach() for m in model.experts]),
                                torch.stack([m.down.weight.detach() for m in model.experts]), top_k=1,
                                activation="relu2")
    x, e, _, _ = batch(model, teacher, generator)
    with torch.no_grad():
        y, parts = model(x, e)
        one = model.mlp(x[5:6], residual=x[5:6])
        ids = torch.empty((32, 1), dtype=torch.int32, device="cuda")
        served = layer(x[:32].contiguous(), ids_out=ids)
    trained = torch.stack([parts[int(e[t])][int((e[:t] == e[t]).sum())] for t in range(32)])
    rel = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())  # noqa: E731
    return {"first_loss": float(losses[0]), "last_loss": float(losses[-1]), "norm": float(norm),
            "one_token": rel(one[0], y[5]), "experts": rel(served, trained),
            "routed": float((ids[:, 0].long() == e[:32]).float().mean())}


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    for k, v in main(ap.parse_args().steps).items():
        print(f"{k}: {v:.4g}")
