"""The layer operators together: NVFP4Linear with bias, activation and residual against the calls it is
made of and against 64-bit gradients, optim.AdamW over a module, and the example that trains a block and
serves it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
import oracle
import workloads
from helpers import log, to_device_bf16

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _layer(d_in, d_out, seed, **kw):
    from bit_block_scaled_quantize_amd.linear import NVFP4Linear
    layer = NVFP4Linear(d_in, d_out, device="cuda", sign_mask=workloads.wgrad_sign_mask(), seed=seed, **kw)
    with torch.no_grad():
        layer.weight.copy_(to_device_bf16(workloads.normal_bf16((d_out, d_in), seed, std=0.05)))
        if layer.bias is not None:
            layer.bias.copy_(torch.randn(d_out, device="cuda"))
    return layer


def _host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("activation", ["none", "relu2", "gelu", "silu"])
@pytest.mark.parametrize("main_grad", [True, False])
def test_layer_is_its_calls(activation, main_grad):
    """Forward and backward give bit for bit what the library calls give, in order."""
    log(f"layer {activation} main_grad={main_grad}")
    layer = _layer(128, 192, 0xC1, bias=True, activation=activation, fp32_main_grad=main_grad)
    x = to_device_bf16(workloads.with_outliers_bf16((64, 128), 5)).requires_grad_(True)
    r = to_device_bf16(workloads.normal_bf16((64, 192), 6)).requires_grad_(True)
    y = layer(x, residual=r)
    dy = to_device_bf16(workloads.normal_bf16((64, 192), 7, std=1e-2))
    y.backward(dy)
    qx, _ = nv.quantize(x.detach())
    qw, qwt = nv.quantize(layer.weight.detach(), "16x16", emit_transposed=True)
    z = torch.empty((64, 192), dtype=torch.bfloat16, device="cuda")
    want = nv.gemm_act(qx, qw, bias=layer.bias.detach(), activation=activation, residual=r.detach(), preact=z)
    assert torch.equal(y.detach(), want)
    assert layer.last_output_amax.item() == want.abs().max().item()
    assert torch.equal(r.grad, dy)
    db = torch.empty((192,), device="cuda")
    dz = nv.act_grad(dy, z, activation=activation, dbias=db)
    mask = layer.sign_mask
    pair = nv.amax_pair(dz, mask)
    qd, _ = nv.quantize(dz, "1x16", "sr", seed=0xC1, offset=0, amax=pair[0:1])
    assert torch.equal(x.grad, nv.gemm_ex(qd, qwt, out_dtype=torch.bfloat16))
    a = nv.rht_quantize(dz, mask, "sr", seed=0xC1, offset=1)
    b = nv.rht_quantize(x.detach(), mask, "rn")
    if main_grad:
        assert torch.equal(layer.main_grad, nv.gemm_ex(a, b)) and layer.weight.grad is None
        assert torch.equal(layer.bias_main_grad, db) and layer.bias.grad is None
    else:
        assert torch.equal(layer.weight.grad, nv.gemm_ex(a, b, out_dtype=torch.bfloat16))
        assert torch.equal(layer.bias.grad, db)


def test_bias_gradient_against_differences():
    """d(sum dY * Y)/d(bias) by central differences of the layer in 64 bits (the quantized product is
    the same at every bias): the step's error is below 1e-6 of the sum of magnitudes; the layer sums
    what act_grad's bound allows, from a pre-activation rounded to BF16 (2^-8 |z|, slope within 2 of it)."""
    log("layer bias gradient")
    for activation in ("relu2", "gelu", "silu", "none"):
        layer = _layer(64, 48, 0xD2, bias=True, activation=activation)
        x = to_device_bf16(workloads.normal_bf16((32, 64), 8)).requires_grad_(True)
        dy = to_device_bf16(workloads.normal_bf16((32, 48), 9))
        layer(x).backward(dy)
        qx, _ = nv.quantize(x.detach())
        qw, _ = nv.quantize(layer.weight.detach(), "16x16")
        p, b, g, h = _host(nv.gemm(qx, qw)), _host(layer.bias), _host(dy), 1e-6
        f = lambda t: (g * oracle.act64(p + b + t, activation)).sum(0)  # noqa: E731
        diff = (f(h) - f(-h)) / (2 * h)
        z = p + b
        tol = (np.abs(g) * (2.0 ** -8 * 2 * np.abs(z) + 1e-4)).sum(0)
        assert np.all(np.abs(_host(layer.bias_main_grad) - diff) <= tol), activation


def test_defaults_are_untouched():
    """Without bias, activation and residual the layer takes the path it had."""
    layer = _layer(64, 32, 3)
    x = to_device_bf16(workloads.normal_bf16((32, 64), 4)).requires_grad_(True)
    y = layer(x)
    assert type(y.grad_fn).__name__.startswith("_LinearFn")
    qx, _ = nv.quantize(x.detach())
    qw, _ = nv.quantize(layer.weight.detach(), "16x16")
    assert torch.equal(y.detach(), nv.gemm_ex(qx, qw, out_dtype=torch.bfloat16))
    with pytest.raises(nv.NVFP4Error, match="multiple of 16"):
        layer(x[:5].detach())


def test_frozen_layer_takes_any_number_of_tokens():
    log("layer frozen")
    layer = _layer(128, 64, 0xE1, bias=True, activation="gelu").freeze()
    x = to_device_bf16(workloads.normal_bf16((33, 128), 2))
    with torch.no_grad():
        for t in (1, 5, 33):
            qx, _ = nv.quantize(x[:t])
            assert torch.equal(layer(x[:t]), nv.gemm_act(qx, layer.frozen, bias=layer.bias, activation="gelu"))
    assert layer.frozen is not None and layer.unfreeze().frozen is None


@pytest.mark.parametrize("states", ["fp32", "8bit"])
def test_optimizer_over_a_module(states):
    from bit_block_scaled_quantize_amd.optim import AdamW
    log(f"optimizer over a module {states}")

    class Net(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.a = _layer(64, 96, 1, bias=True, activation="silu")
            self.b = _layer(96, 32, 2)
            self.norm = torch.nn.Parameter(torch.ones(64, device="cuda"))

    net = Net()
    opt = AdamW.of(net, lr=1e-2, states=states, max_norm=1.0)
    assert len(opt.params) == 4
    for step in range(3):
        x = to_device_bf16(workloads.normal_bf16((32, 64), 20 + step))
        y = net.b(net.a((x.float() * net.norm).bfloat16()))
        y.float().square().mean().backward()
        grads = [g.clone() for g in opt.grads]
        masters = [_host(m) for m in opt.masters]
        norm = opt.step()
        assert abs(norm.item() - np.sqrt(sum(np.square(_host(g)).sum() for g in grads))) <= 1e-5 * norm.item()
        for p, m, before in zip(opt.params, opt.masters, masters):
            assert np.abs(_host(m) - before).max() > 0
            assert torch.equal(p, m.bfloat16() if p.dtype == torch.bfloat16 else m)
        assert net.a.weight_amax.item() == net.a.weight.abs().max().item()
        # the amax from the step makes the next quantization one pass with the same result
        qa, _ = nv.quantize(net.a.weight.detach(), "16x16", amax=net.a.weight_amax)
        qb, _ = nv.quantize(net.a.weight.detach(), "16x16")
        assert torch.equal(qa.codes, qb.codes) and torch.equal(qa.scales, qb.scales)
        opt.zero_grad()
        assert all(torch.count_nonzero(g).item() == 0 for g in opt.grads)
    state = opt.state_dict()
    for g in opt.grads:
        g.fill_(1e-2)
    opt.step()
    after = [m.clone() for m in opt.masters]
    opt.load_state_dict(state)
    assert opt.steps == 3 and net.a.weight_amax is None
    for g in opt.grads:
        g.fill_(1e-2)
    opt.step()
    assert all(torch.equal(a, m) for a, m in zip(after, opt.masters))
    with pytest.raises(nv.NVFP4Error):
        AdamW([(net.norm, None)])
    with pytest.raises(nv.NVFP4Error):
        AdamW([(net.norm, net.norm.grad)], states="4bit")


def test_example():
    """60 steps more than halve the loss; one token alone gives the batch's result up to its own
    tensor scale (one NVFP4 rounding of the activations apart, 2^-2 of an element at worst and some
    10% of the norm); the served experts differ from the trained ones by the activations' rounding."""
    log("example")
    spec = importlib.util.spec_from_file_location("train_and_serve", os.path.join(ROOT, "examples", "train_and_serve.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    r = ex.main(60)
    log(str(r))
    assert r["last_loss"] < 0.5 * r["first_loss"] and np.isfinite(r["norm"])
    assert r["one_token"] < 0.3 and r["experts"] < 0.3
    assert r["routed"] > 0.9
