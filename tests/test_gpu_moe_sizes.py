"""nvfp4_moe_tokens at layer sizes of real use, where K is split over several steps of every wave: a
token's result is bit for bit the same in every batch; and just past the sizes from which the kernels take
another turn: 4096 elements of K staged at a time (and of a token brought to FP16, and of a router's row),
128 maxima of h (ffn 2048), 8 tokens of an expert at a time. Bounds as in test_gpu_moe.py."""
import numpy as np
import pytest
import torch

from helpers import log
from test_gpu_moe import Layer, _bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# K of whole and of ragged 64-element runs; more than four steps of every wave; two stagings of K
INDEPENDENT = [dict(e=6, h=2688, f=1856, k=3), dict(e=5, h=2688, f=1856, k=2, activation="silu", gated=True),
               dict(e=4, h=2704, f=1040, k=2, activation="gelu"), dict(e=3, h=4352, f=4176, k=1),
               dict(e=3, h=5136, f=2064, k=2, activation="silu", gated=True, score="sigmoid")]


@pytest.mark.parametrize("case", INDEPENDENT, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_a_token_does_not_know_the_others(case):
    log(f"moe batches {case}")
    c = dict(case)
    layer = Layer(c.pop("e"), c.pop("h"), c.pop("f"), c.pop("k"), 820, **c)
    x = _bf16((64, layer.h), 821, outliers=True)
    y, ids, w = layer.run(x)
    for first, n in ((0, 1), (63, 1), (7, 2), (20, 4), (3, 5), (40, 8), (9, 17), (0, 33)):
        part = layer.run(x[first:first + n].contiguous())
        assert np.array_equal(part[1], ids[first:first + n]) and np.array_equal(part[2], w[first:first + n])
        assert torch.equal(part[0], y[first:first + n]), f"{n} tokens from {first}"


LARGE = [dict(h=4112, f=2064), dict(h=8208, f=64), dict(h=4096, f=4176, activation="silu", gated=True),
         dict(h=272, f=8208, activation="gelu"), dict(h=4160, f=4112, activation="silu", gated=True, score="sigmoid")]


@pytest.mark.parametrize("t", [1, 4, 5, 20])
@pytest.mark.parametrize("case", LARGE, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_past_one_turn(case, t):
    """Two experts, one a token: more than 8 tokens on one of them at 20."""
    log(f"moe large {case} t={t}")
    c = dict(case)
    layer = Layer(2, c.pop("h"), c.pop("f"), 1, 840, **c)
    x = _bf16((t, layer.h), 841 + t, outliers=True)
    layer.check(x, str(case))
    assert t < 20 or np.bincount(layer.run(x)[1][:, 0]).max() > 8


def test_past_one_turn_with_rows_anywhere():
    """The same walks over x and the router where rows start on any element."""
    log("moe large, strides")
    layer = Layer(2, 4112, 64, 2, 860)
    x = _bf16((3, 4112), 861)
    wide = torch.zeros((3, 4112 + 3), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:4113] = x
    layer.check(wide[:, 1:4113], "strides")


@pytest.mark.parametrize("which", ["w1", "w2"])
@pytest.mark.parametrize("gated", [False, True])
def test_small_scales(which, gated):
    """Tokens and tensor scales whose product leaves FP32's normal range on the way to a result that does
    not: 1e-32 and 2^-26 or so, results of 1e-36."""
    log(f"moe small scales {which} gated={gated}")
    layer = Layer(8, 128, 64, 2, 880, activation="none", gated=gated)
    getattr(layer.gpu.weights, which).global_scale.mul_(2.0 ** -13)
    x = _bf16((6, 128), 881)
    size = 1e-32 ** (0.5 if gated else 1)                            # gated: h is of the order of x^2
    x = (x.float() * (size * torch.tensor([0.7, 1.0, 1.3, 2.0, 3.0, 5.0], device="cuda")[:, None])).bfloat16()
    layer.check(x, "small scales")
