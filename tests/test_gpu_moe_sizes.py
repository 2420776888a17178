"""nvfp4_moe_tokens at layer sizes of real use, where K is split over several steps of every wave: a
token's result is bit for bit the same in every batch."""
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
