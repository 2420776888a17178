"""linear_cross_entropy where the target takes nearly all of a token's probability: the loss is a small difference there.

The logits are exact (a few bits each, one product a logit), so what is tested is the softmax alone.

Bounds. With d = log(sum over the others of exp(l - l[target])), loss = log(1 + exp(d)). An exponent l - top is exact or rounded once,
and its product with log2(e) once (2^-24 of at most 128, each), the exponential itself to 2^-23, the additions of a tile, of the tiles and of the
joins are some 150, of positive terms (2^-24 each), d is rounded twice at a size below 128 (2^-18 each): exp(d) is within 2^-15 of its value, relative, and so is the loss
with a few roundings: held to 2^-14."""
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
from helpers import log

pytestmark = pytest.mark.gpu

LEVELS = [1.0, 4.0, 8.0, 12.0, 15.0, 18.0, 20.0, 21.0, 22.0, 25.0, 28.0, 30.0, 40.0, 60.0, 70.0]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _case(v, h, seed):
    """x, w, targets, grad and the exact logits: token i's target has L = LEVELS[i], every other word L c, c one of 0, -1/8 .. -1."""
    t = len(LEVELS)
    g = torch.Generator().manual_seed(seed)
    level, at = torch.tensor(LEVELS), torch.arange(t)
    x, w = torch.zeros(t, h), torch.zeros(v, h)
    tg = torch.randperm(v, generator=g)[:t]
    x[:, 0] = level
    w[:, 0] = torch.randint(-8, 1, (v,), generator=g) / 8.0
    w[tg, 0] = 0.0
    x[at, 2 + at] = 1.0                                       # dW's column 2 + i: token i's G
    x[at, 2 + t + at] = level                                 # the target's logit; dx's column 2 + t + i: its G
    w[tg, 2 + t + at] = 1.0
    return [a.cuda() for a in (x.bfloat16(), w.bfloat16(), tg, torch.rand((t,), generator=g) + 0.5)], (x.double() @ w.double().t()).cuda()


def _want(logits, tg, grad):
    """(loss, G) in 64 bits without cancellation."""
    at = torch.arange(logits.shape[0], device="cuda")
    d = logits - logits[at, tg][:, None]
    G = d.clone()
    d[at, tg] = -torch.inf
    loss = torch.logaddexp(torch.logsumexp(d, 1), torch.zeros((), dtype=torch.float64, device="cuda"))
    G = torch.exp(G - loss[:, None])
    G[at, tg] = torch.expm1(-loss)
    return loss, G * grad.double()[:, None]


@pytest.mark.parametrize("v,h", [(16, 48), (40, 64), (300, 64), (3001, 48), (70001, 64)])
def test_loss_of_confident_tokens(v, h):
    (x, w, tg, grad), logits = _case(v, h, v)
    log(f"confident loss {v} words, hidden {h}")
    loss, lse = nv.linear_cross_entropy(x, w, tg)
    want, _ = _want(logits, tg, grad)
    off = (loss.double() - want).abs() / want
    assert float(off.max()) <= 2.0 ** -14, (off.tolist(), want.tolist())
    assert bool(((lse.double() - torch.logsumexp(logits, 1)).abs() <= 2.0 ** -18 + 2.0 ** -14 * want).all())
    # tokens that do not count have the same lse, to its rounding
    none = nv.linear_cross_entropy(x, w, torch.full_like(tg, -100))
    assert not none[0].any() and bool(((none[1] - lse).abs() <= 2.0 ** -16 + 2.0 ** -14 * loss).all())


def test_one_word_and_words_alike():
    x = torch.randn(33, 32, device="cuda").bfloat16()
    tg = torch.zeros(33, dtype=torch.int64, device="cuda")
    loss, lse = nv.linear_cross_entropy(x, x[:1].contiguous(), tg)
    assert not loss.any() and float((lse - (x.float() @ x[0].float())).abs().max()) <= 1e-4
    w = x[:1].expand(5, 32).contiguous()                      # five words alike: log 5 each
    loss, lse = nv.linear_cross_entropy(x, w, tg + 3)
    assert float((loss.double() - torch.log(torch.tensor(5.0, dtype=torch.float64))).abs().max()) <= 2.0 ** -20


def test_infinite_and_huge_logits():
    """The largest logits that FP32 holds; a target at -inf has an infinite loss, one at +inf none that is a number."""
    x = torch.zeros(3, 16, device="cuda")
    w = torch.zeros(20, 16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = 2.0 ** 64, 2.0 ** 100, 2.0 ** 100
    w[3, 0], w[4, 0] = 2.0 ** 63.5, -2.0 ** 100
    x, w = x.bfloat16(), w.bfloat16()
    tg = torch.tensor([3, 4, 5], device="cuda")
    loss, lse = nv.linear_cross_entropy(x, w, tg)
    torch.cuda.synchronize()
    assert float(loss[0]) == 0.0 and float(lse[0]) == float((x[0].float() * w[3].float())[0]) and torch.isfinite(lse[0])
    assert not torch.isfinite(loss[1]) and not torch.isfinite(loss[2])
