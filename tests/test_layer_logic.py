"""What NVFP4Linear and optim.AdamW do with their buffers, on the CPU: the library calls are stood in for
by plain products (no quantization) and the optimizer's step by the 64-bit oracle, so that only the
wrappers' own decisions are tested: which gradients are computed, where they go, what is stepped."""
import numpy as np
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
import oracle
from bit_block_scaled_quantize_amd import linear, optim
from bit_block_scaled_quantize_amd.linear import NVFP4Linear
from bit_block_scaled_quantize_amd.optim import AdamW


class Plan:
    """AdamWPlan without a device table."""

    def __init__(self, tensors):
        self.tensors, self.device = list(tensors), torch.device("cpu")


def _adamw(plan, lr, betas, eps, step, max_norm=None, seed=0, amax_out=None, **_):
    norm = np.sqrt(sum(float(t.grad.double().square().sum()) for t in plan.tensors))
    clip = 1.0 if max_norm is None else min(1.0, max_norm / (norm + 1e-6))
    for i, t in enumerate(plan.tensors):
        out = oracle.adamw64(t.p.reshape(-1).numpy(), t.grad.reshape(-1).float().numpy(), t.m.numpy(), t.v.numpy(), lr,
                             *betas, eps, step, t.weight_decay, clip)
        for dst, src in zip((t.p, t.m, t.v), out):
            dst.numpy().reshape(-1)[:] = src                 # as the kernel writes: no version counter moves
        w = t.p if t.w_out is None else t.w_out
        if t.w_out is not None:
            t.w_out.view(torch.int16).numpy().reshape(-1)[:] = t.p.bfloat16().view(torch.int16).numpy().reshape(-1)
        if amax_out is not None:
            amax_out[i] = w.abs().max().float()
    return None if max_norm is None else torch.tensor([norm])


@pytest.fixture(autouse=True)
def library(monkeypatch):
    """The calls made, by name, in order."""
    calls = []

    def quantize(x, block="1x16", rnd="rn", amax=None, emit_transposed=False, **kw):
        calls.append(("quantize", amax))
        return x.detach().float().clone(), x.detach().t().float().clone() if emit_transposed else None

    def gemm_ex(a, b, out=None, accumulate=False, out_dtype=torch.float32, amax_out=None):
        d = a @ b.t()
        if accumulate:
            return out.add_(d)
        if amax_out is not None:
            amax_out.copy_(d.abs().max())
        return d.to(out_dtype)

    def gemm_act(a, b, bias=None, activation="none", residual=None, preact=None, amax_out=None):
        z = a @ b.t() + (0 if bias is None else bias)
        if preact is not None:
            preact.copy_(z)
        d = {"none": z, "relu2": z.clamp_min(0).square()}[activation] + (0 if residual is None else residual)
        amax_out.copy_(d.abs().max())
        return d.bfloat16()

    def act_grad(dy, preact=None, activation="none", dbias=None, accumulate=False, bias_only=False):
        g = dy.float() * (2 * preact.float().clamp_min(0) if activation == "relu2" else 1)
        if dbias is not None:
            dbias.copy_(g.sum(0) + (dbias if accumulate else 0))
        return None if bias_only else g.bfloat16()

    def rht_quantize(x, *_, **__):
        calls.append(("rht_quantize", None))
        return x.detach().t().float()

    for name, fn in dict(quantize=quantize, gemm_ex=gemm_ex, gemm_act=gemm_act, act_grad=act_grad, rht_quantize=rht_quantize,
                         amax=lambda x, **_: x.abs().max().float().reshape(1),
                         amax_pair=lambda x, _: x.abs().max().float().expand(2).clone()).items():
        monkeypatch.setattr(linear, name, fn)
    monkeypatch.setattr(optim, "AdamWPlan", Plan)
    monkeypatch.setattr(optim, "adamw", _adamw)
    return calls


def _layer(d_in, d_out, seed, **kw):
    torch.manual_seed(seed)
    layer = NVFP4Linear(d_in, d_out, **kw)
    with torch.no_grad():
        layer.weight.copy_(torch.randn(d_out, d_in) * 0.2)
        if layer.bias is not None:
            layer.bias.copy_(torch.randn(d_out))
    return layer


def _x(rows, cols, seed=0):
    torch.manual_seed(100 + seed)
    return torch.randn(rows, cols).bfloat16()


@pytest.mark.parametrize("kw", [dict(), dict(bias=True, activation="relu2")], ids=["plain", "act"])
def test_a_frozen_layer_is_left_alone(kw):
    """requires_grad_(False) between trainable layers: no gradient is added to the layer's buffers, the
    optimizer does not step or decay it, and its gradient is no part of the norm."""
    net = torch.nn.Sequential(_layer(32, 48, 1, **kw), _layer(48, 64, 2, **kw), _layer(64, 32, 3, **kw))
    net[1].requires_grad_(False)
    net[1].main_grad.fill_(0.5)                                       # of an earlier step: not to be read either
    keep = [t.clone() for t in net[1].parameters()]
    opt = AdamW.of(net, lr=1e-2, weight_decay=0.1, max_norm=1.0)
    addresses = {p.data_ptr() for p in opt.params}
    assert not addresses & {p.data_ptr() for p in net[1].parameters()}
    assert addresses == {p.data_ptr() for p in net.parameters() if p.requires_grad}
    for _ in range(2):
        net(_x(32, 32)).float().square().mean().backward()
        norm = opt.step()
        assert norm.item() == pytest.approx(np.sqrt(sum(float(g.double().square().sum()) for g in opt.grads)))
        assert all(torch.count_nonzero(g) for g in opt.grads)
        opt.zero_grad()
    assert torch.all(net[1].main_grad == 0.5)
    if net[1].bias is not None:
        assert torch.count_nonzero(net[1].bias_main_grad).item() == 0
    assert all(torch.equal(a, b) for a, b in zip(net[1].parameters(), keep))


@pytest.mark.parametrize("frozen", ["weight", "bias"])
def test_one_of_weight_and_bias_frozen(frozen):
    layer = _layer(32, 48, 4, bias=True, activation="relu2")
    getattr(layer, frozen).requires_grad_(False)
    x = _x(16, 32, 4).requires_grad_(True)
    layer(x).float().sum().backward()
    assert torch.count_nonzero(x.grad) > 0
    got = {"weight": layer.main_grad, "bias": layer.bias_main_grad}
    for name, g in got.items():
        assert (torch.count_nonzero(g).item() == 0) == (name == frozen)
    assert len(AdamW.of(layer).params) == 1


class Tied(torch.nn.Module):
    """Two layers with one weight, and (table) the weight as an ordinary parameter too."""

    def __init__(self, second_main_grad=True, table=False, bias=False):
        super().__init__()
        self.a = _layer(32, 32, 5, bias=bias)
        self.b = _layer(32, 32, 6, bias=bias, fp32_main_grad=second_main_grad)
        self.b.weight = self.a.weight
        if bias:
            self.b.bias = self.a.bias
        self.table = table

    def forward(self, x):
        y = self.b(self.a(x))
        return y + x @ self.a.weight.t() if self.table else y


def _weight_gradient(net, x):
    """The gradient of the tied weight and bias summed over all of their uses, in FP32."""
    w = net.a.weight.detach().float().requires_grad_(True)
    b = (torch.zeros(32) if net.a.bias is None else net.a.bias.detach().clone()).requires_grad_(True)
    h = (x.float() @ w.t() + b).bfloat16().float()
    y = (h @ w.t() + b).bfloat16().float()
    y = y + (x.float() @ w.t() if net.table else 0)
    y.sum().backward()
    return w.grad, b.grad


@pytest.mark.parametrize("kw", [dict(), dict(bias=True), dict(second_main_grad=False), dict(table=True),
                                dict(second_main_grad=False, table=True)],
                         ids=lambda k: "-".join(k) or "plain")
@pytest.mark.parametrize("backward_before", [False, True], ids=["", "gradients-before"])
def test_tied_weights_get_every_gradient(kw, backward_before):
    """Each use of a shared weight adds to the gradient that is stepped, whichever buffer it goes to,
    also where a backward pass came before the optimizer; nothing of it is left for the next step.
    BF16 gradients: 2^-8 of the sum of magnitudes over 16 rows, three uses."""
    net = Tied(**kw)
    x = _x(16, 32, 7)
    want, want_bias = _weight_gradient(net, x)
    if backward_before:
        net(x).float().sum().backward()
    opt = AdamW.of(net, lr=1e-2, max_norm=1e9, weight_decay=0.0)
    assert len(opt.params) == (1 if net.a.bias is None else 2)
    for step in range(2):
        if step or not backward_before:
            net(x).float().sum().backward()
        want, want_bias = _weight_gradient(net, x)
        norm = opt.step()
        tol = 2.0 ** -7 * float(want.abs().max())
        assert torch.allclose(opt.grads[0], want, rtol=0, atol=3 * tol)
        if net.a.bias is not None:
            assert torch.allclose(opt.grads[1], want_bias, rtol=0, atol=2.0 ** -7 * float(want_bias.abs().max()))
        assert norm.item() == pytest.approx(np.sqrt(sum(float(g.double().square().sum()) for g in opt.grads)))
        assert net.a.weight_amax.item() == net.a.weight.abs().max().item()
        assert net.b.weight_amax is None or net.b.weight_amax.item() == net.a.weight_amax.item()
        opt.zero_grad()
        for layer in (net.a, net.b):
            assert all(g is None or torch.count_nonzero(g).item() == 0
                       for g in (layer.main_grad, layer.bias_main_grad, layer.weight.grad))


class Scaled(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.norm = torch.nn.Parameter(torch.ones(32))
        self.lin = _layer(32, 32, 8, bias=True)

    def forward(self, x):
        return self.lin((x.float() * self.norm).bfloat16())


def _moved_grad(net):
    net.norm.grad = net.norm.grad.clone()


def _no_grad(net):
    net.zero_grad()                                                   # set_to_none is torch's default


def _moved_main(net):
    net.lin.main_grad = torch.zeros_like(net.lin.main_grad)


def _moved_bias_main(net):
    net.lin.bias_main_grad = torch.zeros_like(net.lin.bias_main_grad)


def _moved_weight(net):
    net.lin.weight.data = net.lin.weight.data.clone()


def _moved_parameter(net):
    net.norm.data = net.norm.data.clone()


@pytest.mark.parametrize("move", [_moved_grad, _no_grad, _moved_main, _moved_bias_main, _moved_weight, _moved_parameter])
def test_a_step_from_buffers_that_moved_is_refused(move):
    """The plan holds addresses: a step from the old gradient, or of the old weight, is an error and
    changes nothing."""
    net = Scaled()
    opt = AdamW.of(net, lr=1e-2)
    net(_x(16, 32, 8)).float().sum().backward()
    opt.step()
    opt.zero_grad()
    move(net)
    net(_x(16, 32, 9)).float().sum().backward()
    keep = [t.clone() for t in opt.masters]
    with pytest.raises(nv.NVFP4Error, match="moved"):
        opt.step()
    assert opt.steps == 1 and all(torch.equal(a, b) for a, b in zip(keep, opt.masters))


def test_gradients_given_one_by_one_are_the_callers():
    """Entries name any gradient; one that is the parameter's .grad has to stay it."""
    p, g = torch.nn.Parameter(torch.ones(8)), torch.full((8,), 0.5)
    opt = AdamW([(p, g)], lr=1e-2)
    opt.step()
    assert p.grad is None and torch.all(p.detach() < 1)
    p.grad = torch.zeros(8)
    opt.step()
    q = torch.nn.Parameter(torch.ones(8))
    q.grad = torch.ones(8)
    opt = AdamW([(q, q.grad)], lr=1e-2)
    opt.step()
    q.grad = None
    with pytest.raises(nv.NVFP4Error, match="moved"):
        opt.step()


def _copy(layer):
    with torch.no_grad():
        layer.weight.copy_(layer.weight * 8)


def _load(layer):
    layer.load_state_dict({k: v * 8 for k, v in layer.state_dict().items()})


def _replace(layer):
    layer.weight.data = layer.weight.data * 8


def _reset(layer):
    torch.nn.init.normal_(layer.weight, std=3.0)


CHANGES = [_copy, _load, _replace, _reset]


@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("kw", [dict(), dict(bias=True)], ids=["plain", "act"])
def test_a_changed_weight_is_not_scaled_by_its_old_maximum(library, change, kw):
    layer = _layer(32, 32, 11, **kw)
    opt = AdamW.of(layer, lr=1e-2)
    x = _x(16, 32, 11)
    layer(x).float().sum().backward()
    opt.step()
    after = layer.weight_amax
    assert after.item() == layer.weight.abs().max().item()
    del library[:]
    layer(x)
    assert [a for n, a in library if n == "quantize"][1] is after     # of X, then of W: one pass
    change(layer)
    assert layer.weight_amax is None
    del library[:]
    layer(x)
    assert [a for n, a in library if n == "quantize"][1] is None
    layer.weight_amax = layer.weight.detach().abs().max().float().reshape(1)
    assert layer.weight_amax.item() == layer.weight.abs().max().item()
    layer.weight_amax = None
    assert layer.weight_amax is None


def test_a_step_counts_as_a_change_of_what_it_writes():
    """The kernel writes behind torch's back: the version counters of the parameters move all the same."""
    net = Scaled()
    opt = AdamW.of(net, lr=1e-2)
    y = net(_x(16, 32, 12)).float().sum() + net.norm.square().sum()   # the square's backward needs norm as it was
    y.backward(retain_graph=True)
    before = [p._version for p in net.parameters()]
    opt.step()
    assert all(p._version > v for p, v in zip(net.parameters(), before))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_a_layer_made_in_inference_mode():
    with torch.inference_mode():
        layer = _layer(32, 32, 13)
        layer.weight_amax = layer.weight.abs().max().float().reshape(1)
        assert layer(_x(16, 32, 13)).shape == (16, 32)
        assert layer.weight_amax is not None


@pytest.mark.parametrize("change", CHANGES + ["step"])
@pytest.mark.parametrize("kw", [dict(), dict(bias=True, activation="relu2")], ids=["plain", "act"])
def test_a_frozen_quantization_follows_the_weight(library, change, kw):
    """freeze() saves the quantization of an unchanged weight and no more than that."""
    layer = _layer(32, 32, 14, **kw)
    opt = AdamW.of(layer, lr=1e-1)
    x = _x(16, 32, 14)
    layer.freeze()

    def calls():
        del library[:]
        with torch.no_grad():
            y = layer(x)
        return y, [n for n, _ in library].count("quantize")

    first, n = calls()
    assert n == 1 and calls()[1] == 1                                 # of X alone
    if change == "step":
        layer(x).float().sum().backward()
        opt.step()
    else:
        change(layer)
    y, n = calls()
    assert n == 2 and not torch.equal(y, first)
    assert calls()[1] == 1 and torch.equal(calls()[0], y)
    layer.unfreeze()
    assert torch.equal(layer(x).detach(), y)


@pytest.mark.parametrize("change", [_copy, _load, _reset])
def test_a_step_starts_from_the_weights_that_are_there(change):
    """Weights loaded after the optimizer was made are stepped, not overwritten by its master copies;
    what was not changed keeps the master's FP32 value (an average swapped in and out again)."""
    layer = _layer(32, 32, 15)
    opt = AdamW.of(layer, lr=1e-3, weight_decay=0.0)
    for seed in range(2):
        layer(_x(16, 32, seed)).float().sum().backward()
        opt.step()
        opt.zero_grad()
    master = opt.masters[0].clone()
    assert not torch.equal(master, master.bfloat16().float())
    keep = layer.weight.detach().clone()
    change(layer)                                                     # swapped in, and out again
    with torch.no_grad():
        layer.weight.copy_(keep)
    assert torch.equal(opt.state_dict()["masters"][0], master)
    change(layer)
    with torch.no_grad():
        layer.weight[:3] = keep[:3]
    here = layer.weight.detach().float()
    here[:3] = master[:3]
    assert torch.equal(opt.state_dict()["masters"][0], here)
    layer(_x(16, 32, 3)).float().sum().backward()
    opt.step()
    assert (opt.masters[0] - here).abs().max() <= 1.5e-2             # a few times lr / (1 - beta1) at most
    assert torch.equal(layer.weight.detach(), opt.masters[0].bfloat16())


def test_a_state_of_other_shapes_is_refused():
    """Before anything of it is copied: one element would spread over a whole tensor."""
    def make(n):
        p = torch.nn.Parameter(torch.full((n,), 2.0))
        return AdamW([(p, torch.ones(n)), (torch.nn.Parameter(torch.full((4,), 3.0)), torch.ones(4))], lr=1e-2)

    opt, other = make(8), make(1)
    opt.step()
    keep = opt.state_dict()
    for key, value in (("masters", other.masters), ("m", other.state_dict()["m"]), ("v", keep["v"][:1])):
        with pytest.raises(nv.NVFP4Error, match="another optimizer"):
            opt.load_state_dict({**keep, "masters": [torch.zeros_like(m) for m in keep["masters"]], key: value})
        assert all(torch.equal(a, b) for k in ("masters", "m", "v") for a, b in zip(opt.state_dict()[k], keep[k])), key
    opt.load_state_dict(keep)


def test_a_refused_step_is_not_counted(monkeypatch):
    p = torch.nn.Parameter(torch.ones(8))
    opt = AdamW([(p, torch.ones(8))], lr=1e-2)
    opt.step()

    def refuse(*_, **__):
        raise nv.NVFP4Error("out of range")

    monkeypatch.setattr(optim, "adamw", refuse)
    with pytest.raises(nv.NVFP4Error):
        opt.step(lr=float("nan"))
    assert opt.steps == 1


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_parameter_named_twice_is_refused(dtype):
    """Two entries of one tensor would step it twice at once, or from two masters."""
    p = torch.nn.Parameter(torch.ones(8, dtype=dtype))
    with pytest.raises(nv.NVFP4Error, match="twice"):
        AdamW([(p, torch.ones(8)), (p, torch.ones(8))])
    empty = torch.nn.Parameter(torch.ones(0, dtype=dtype))
    AdamW([(empty, torch.ones(0)), (torch.nn.Parameter(torch.ones(0)), torch.ones(0)), (p, torch.ones(8))])


@pytest.mark.parametrize("name", ["weight", "bias"])
def test_a_step_of_a_parameter_that_its_layer_no_longer_has_is_refused(name):
    """load_state_dict(assign=True) and the like put other parameters in the layer's place."""
    layer = _layer(32, 32, 16, bias=True)
    opt = AdamW.of(layer)
    opt.step()
    layer.load_state_dict({k: v.clone() if k == name else v for k, v in layer.state_dict(keep_vars=True).items()}, assign=True)
    with pytest.raises(nv.NVFP4Error, match=f"{name}.*moved"):
        opt.step()
    assert opt.steps == 1
