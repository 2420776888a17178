"""linear_cross_entropy and its gradient where the target takes nearly all of a token's probability: the loss and the target's
G = grad (p - 1) are small differences there.

The logits are exact (a few bits each, one product a logit), so what is tested is the softmax alone. Every token has a column of x in
which dW holds that token's G by itself, and one of w in which dx holds its target's G.

Bounds. With d = log(sum over the others of exp(l - l[target])), loss = log(1 + exp(d)). An exponent l - top is exact or rounded once,
and its product with log2(e) once (2^-24 of at most 128, each), the exponential itself to 2^-23, the additions of a tile, of the tiles and of the
joins are some 150, of positive terms (2^-24 each), d is rounded twice at a size below 128 (2^-18 each): exp(d) is within 2^-15 of its value, relative, and so is the loss
and 1 - p = 1 - exp(-loss), with a few roundings: held to 2^-14. G's other entries: exp(l - lse) with lse rounded (2^-24 of at most 128) and BF16: 2^-8 + 2^-16.
dx and a BF16 dW: one rounding more, 2^-8; an FP32 dW of the target: its G's BF16 remainder in BF16, 2^-16."""
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
from bit_block_scaled_quantize_amd.loss import LinearCrossEntropy
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


@pytest.mark.parametrize("v,h", [(16, 48), (300, 64), (3001, 48), (70001, 64)])
def test_gradient_of_confident_tokens(v, h):
    (x, w, tg, grad), logits = _case(v, h, v)
    log(f"confident gradient {v} words, hidden {h}")
    t = x.shape[0]
    at = torch.arange(t, device="cuda")
    loss, lse = nv.linear_cross_entropy(x, w, tg)
    _, G = _want(logits, tg, grad)
    d32 = torch.empty((v, h), device="cuda")
    dx, _ = nv.linear_cross_entropy_grad(x, w, tg, lse, grad, dweight=d32, loss=loss)
    _, dw = nv.linear_cross_entropy_grad(x, w, tg, lse, grad, need_dx=False, loss=loss)
    own = G[at, tg]
    got = d32[:, 2:2 + t].double().t()                        # G
    off = (got[at, tg] - own).abs() / own.abs()
    assert float(off.max()) <= 2.0 ** -14 + 2.0 ** -15, (off.tolist(), own.tolist())
    rest = torch.ones_like(G, dtype=torch.bool)
    rest[at, tg] = False
    normal = rest & (G.abs() > 2.0 ** -120)
    assert float(((got - G).abs() / G.abs().clamp_min(1e-300))[normal].max()) <= 2.0 ** -8 + 2.0 ** -15
    assert bool(((dx[at, 2 + t + at].double() - own).abs() <= (2.0 ** -8 + 2.0 ** -13) * own.abs()).all())
    b = dw[:, 2:2 + t].double().t()
    assert bool(((b[at, tg] - own).abs() <= (2.0 ** -8 + 2.0 ** -13) * own.abs()).all())


def test_gradient_from_lse_alone():
    """Without the loss p - 1 comes from the difference to lse: off by what lse was rounded by (half a step at its size) and 2^-14 of
    itself, but by nothing more."""
    (x, w, tg, grad), logits = _case(3001, 48, 5)
    t = x.shape[0]
    at = torch.arange(t, device="cuda")
    _, lse = nv.linear_cross_entropy(x, w, tg)
    d32 = torch.empty((3001, 48), device="cuda")
    nv.linear_cross_entropy_grad(x, w, tg, lse, grad, dweight=d32, need_dx=False)
    got = d32[:, 2:2 + t].t()[at, tg].double()
    # the definition with this lse
    l = logits[at, tg]
    want = torch.expm1(l - lse.double()) * grad.double()
    assert bool(((got - want).abs() <= 2.0 ** -14 * want.abs()).all()), (got.tolist(), want.tolist())


def test_module_of_confident_tokens():
    (x, w, tg, grad), logits = _case(3001, 48, 6)
    t = x.shape[0]
    at = torch.arange(t, device="cuda")
    head = LinearCrossEntropy(48, 3001, device="cuda", reduction="none")
    head.weight.data.copy_(w)
    loss = head(x.requires_grad_(), tg)
    loss.backward(grad)
    want, G = _want(logits, tg, grad)
    assert float(((loss.double() - want).abs() / want).max()) <= 2.0 ** -14
    got = head.main_grad[:, 2:2 + t].t()[at, tg].double()
    assert bool(((got - G[at, tg]).abs() <= (2.0 ** -14 + 2.0 ** -15) * G[at, tg].abs()).all())


def test_one_word_and_words_alike():
    x = torch.randn(33, 32, device="cuda").bfloat16()
    tg = torch.zeros(33, dtype=torch.int64, device="cuda")
    loss, lse = nv.linear_cross_entropy(x, x[:1].contiguous(), tg)
    assert not loss.any() and float((lse - (x.float() @ x[0].float())).abs().max()) <= 1e-4
    w = x[:1].expand(5, 32).contiguous()                      # five words alike: log 5 each
    loss, lse = nv.linear_cross_entropy(x, w, tg + 3)
    assert float((loss.double() - torch.log(torch.tensor(5.0, dtype=torch.float64))).abs().max()) <= 2.0 ** -20
    dx, dw = nv.linear_cross_entropy_grad(x, w, tg + 3, lse, torch.ones(33, device="cuda"), loss=loss)
    assert torch.isfinite(dx.float()).all() and torch.isfinite(dw.float()).all()


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


def test_refuses_a_loss_of_another_kind():
    (x, w, tg, grad), _ = _case(40, 48, 1)
    loss, lse = nv.linear_cross_entropy(x, w, tg)
    for bad in (loss[:3], loss.double(), loss.cpu()):
        with pytest.raises(nv.NVFP4Error, match="loss"):
            nv.linear_cross_entropy_grad(x, w, tg, lse, grad, loss=bad)


def test_the_loss_that_a_caller_gets_may_be_changed():
    (x, w, tg, grad), logits = _case(40, 48, 1)
    head = LinearCrossEntropy(48, 40, device="cuda", reduction="none", fp32_main_grad=False)
    head.weight.data.copy_(w)
    a = head(x.requires_grad_(), tg)
    a.backward(grad)
    want = x.grad.clone()
    x.grad = None
    b = head(x, tg)
    b.detach().zero_()
    b.mul_(2.0)
    b.backward(grad / 2)
    assert torch.equal(x.grad, want)


def test_tokens_that_lean_to_their_targets():
    """Logits of real products, target logits from 5 to 60. A logit is off by at most e = 1e-5 of its addends' sizes (the library's bound
    for an FP32 product), a difference of two by 2 e, so the loss and 1 - p by a factor exp(2 e), besides the bounds above."""
    t, h, v = 60, 256, 3001
    g = torch.Generator().manual_seed(3)
    w, tg = torch.randn(v, h, generator=g) * h ** -0.5, torch.randperm(v, generator=g)[:t]
    x = w[tg] * torch.linspace(5, 60, t)[:, None]
    x, w = torch.cat([x, torch.eye(t)], 1).bfloat16(), torch.cat([w, torch.zeros(v, t)], 1).bfloat16()
    x, w = (torch.nn.functional.pad(m, (0, -(h + t) % 16)).cuda() for m in (x, w))
    tg, grad, at = tg.cuda(), torch.ones(t, device="cuda"), torch.arange(t, device="cuda")
    logits = x.double() @ w.double().t()
    want, G = _want(logits, tg, grad)
    assert float(want.min()) < 1e-9 and float(want.max()) > 1
    e = 1e-5 * float((x.double().abs() @ w.double().abs().t()).max())
    rel = float(torch.expm1(torch.tensor(2 * e))) + 2.0 ** -14
    assert rel < 0.01
    loss, lse = nv.linear_cross_entropy(x, w, tg)
    assert bool(((loss.double() - want).abs() <= rel * want).all())
    d32 = torch.empty(w.shape, device="cuda")
    nv.linear_cross_entropy_grad(x, w, tg, lse, grad, dweight=d32, need_dx=False, loss=loss)
    own = G[at, tg]
    assert bool(((d32[tg, h + at].double() - own).abs() <= (rel + 2.0 ** -15) * own.abs()).all())


def test_module_without_gradients(monkeypatch):
    """Evaluation: the same losses, and no copy of them is kept for a backward pass."""
    (x, w, tg, grad), _ = _case(40, 48, 1)
    head = LinearCrossEntropy(48, 40, device="cuda", reduction="none")
    head.weight.data.copy_(w)
    want = head(x, tg).detach().clone()
    copies, clone = [], torch.Tensor.clone
    monkeypatch.setattr(torch.Tensor, "clone", lambda t, **kw: copies.append(t.shape) or clone(t, **kw))
    with torch.no_grad():
        got = head(x, tg)
    assert torch.equal(got, want) and not copies
    head(x, tg)
    assert len(copies) == 1
    head.weight.requires_grad_(False)
    assert torch.equal(head(x, tg), want) and len(copies) == 1
