"""What NVFP4Linear, optim.AdamW and moe.MoETokens keep between calls, on the GPU: a layer gives the
result of the weights it has at the call, however they came there."""
import numpy as np
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
import workloads
from bit_block_scaled_quantize_amd.linear import NVFP4Linear
from bit_block_scaled_quantize_amd.optim import AdamW
from helpers import log, to_device_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _layer(d_in, d_out, seed, **kw):
    layer = NVFP4Linear(d_in, d_out, device="cuda", sign_mask=workloads.wgrad_sign_mask(), seed=seed, **kw)
    with torch.no_grad():
        layer.weight.copy_(_bf16((d_out, d_in), seed, 0.05))
        if layer.bias is not None:
            layer.bias.copy_(torch.randn(d_out, device="cuda"))
    return layer


def _bf16(shape, seed, std=1.0):
    return to_device_bf16(workloads.normal_bf16(shape, seed, std=std))


def _fresh(layer, x):
    """The layer's result by the library's calls, nothing kept."""
    qx, _ = nv.quantize(x)
    qw, _ = nv.quantize(layer.weight.detach(), "16x16")
    if layer.bias is None and layer.activation == "none":
        return nv.gemm_ex(qx, qw, out_dtype=torch.bfloat16)
    return nv.gemm_act(qx, qw, bias=None if layer.bias is None else layer.bias.detach(), activation=layer.activation)


@pytest.mark.parametrize("kw", [dict(), dict(bias=True, activation="gelu")], ids=["plain", "act"])
def test_weights_loaded_after_a_step(kw):
    log(f"layer state {kw}")
    layer = _layer(128, 96, 21, **kw)
    opt = AdamW.of(layer, lr=1e-2)
    x = _bf16((32, 128), 22)
    layer(x).float().sum().backward()
    opt.step()
    assert torch.equal(layer(x).detach(), _fresh(layer, x))
    layer.load_state_dict({k: v * 16 for k, v in layer.state_dict().items()})     # far above the step's maximum
    assert torch.equal(layer(x).detach(), _fresh(layer, x))
    opt.zero_grad()
    layer(x).float().sum().backward()
    opt.step()
    assert layer.weight_amax.item() == layer.weight.abs().max().item()
    assert torch.equal(layer(x).detach(), _fresh(layer, x))


def test_a_frozen_layer_after_a_step():
    """An evaluation between two steps uses the weights of the last one, for one token too."""
    log("frozen layer after a step")
    layer = _layer(128, 96, 23, bias=True, activation="silu")
    opt = AdamW.of(layer, lr=3e-1)
    x = _bf16((32, 128), 24)
    layer.freeze()
    for _ in range(3):
        with torch.no_grad():
            for t in (1, 7, 32):
                assert torch.equal(layer(x[:t]), _fresh(layer, x[:t]))
        layer(x).float().sum().backward()
        opt.step()
        opt.zero_grad()


@pytest.mark.parametrize("states", ["fp32", "8bit"])
def test_a_step_after_loading_weights(states):
    """The step moves the loaded weights by what it moves any weights with this gradient and history, not
    back to those of the optimizer's master copies."""
    log(f"step after loading {states}")
    layer = _layer(64, 48, 25)
    opt = AdamW.of(layer, lr=1e-2, weight_decay=0.0, states=states)
    layer.main_grad.copy_(_bf16((48, 64), 26).float())
    opt.step()
    loaded = _bf16((48, 64), 27, 4.0)
    layer.load_state_dict({"weight": loaded})
    opt.step()
    moved = (opt.masters[0] - loaded.float()).abs()
    assert torch.equal(layer.weight.detach(), opt.masters[0].bfloat16())
    # the same gradient twice: m/(1 - b1^t) = g and v/(1 - b2^t) = g^2, 8-bit states within two E4M3 gaps (2^-3 each)
    assert moved.max().item() <= 1e-2 * 1.5 and moved.min().item() >= 1e-2 * 0.5


def _fill_freed_memory():
    """Hands out, and writes, blocks of the sizes that a small layer's tensors have."""
    kept = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (512, 1024, 4096, 8192, 16384, 32768) for _ in range(40)]
    torch.cuda.synchronize()
    return kept


def test_an_expert_layer_keeps_the_tensors_it_was_made_with():
    """Also where its weights are given other tensors later: the addresses it passes stay valid."""
    from bit_block_scaled_quantize_amd.moe import MoETokens
    log("expert layer's tensors")
    make = lambda seed: MoETokens.from_bf16(_bf16((8, 128), seed), _bf16((8 * 64, 128), seed + 1, 0.1).view(8, 64, 128),  # noqa: E731
                                            _bf16((8 * 128, 64), seed + 2, 0.1).view(8, 128, 64), 2)
    layer, other = make(31), make(41)
    x = _bf16((5, 128), 34)
    want = layer(x).clone()
    torch.cuda.synchronize()
    layer.weights.router, layer.weights.w1, layer.weights.w2 = other.weights.router, other.weights.w1, other.weights.w2
    del other
    held = _fill_freed_memory()
    assert torch.equal(layer(x), want)
    del held


def test_a_plan_keeps_the_tensors_it_was_made_with():
    log("plan's tensors")
    def tensors():
        return [nv.AdamWTensor(p=_bf16((16, 64), 51).float().reshape(-1), grad=_bf16((16, 64), 52).float().reshape(-1),
                               m=torch.zeros(1024, device="cuda"), v=torch.zeros(1024, device="cuda"))]
    want = tensors()
    nv.adamw(nv.AdamWPlan(want), lr=1e-2, step=1)
    ts = tensors()
    plan, p = nv.AdamWPlan(ts), ts[0].p
    torch.cuda.synchronize()
    ts[0].grad = ts[0].m = ts[0].v = None
    plan.tensors[0].p = None
    plan.tensors.clear()
    held = _fill_freed_memory()
    nv.adamw(plan, lr=1e-2, step=1)
    assert torch.equal(p, want[0].p) and all(torch.all(h == 0x5A) for h in held)


def test_the_first_call_of_an_expert_layer_on_another_stream():
    """The workspace's counters are zero by then, however busy the stream is that the layer was made on."""
    from bit_block_scaled_quantize_amd.moe import MoETokens
    log("expert layer's first call")
    w = MoETokens.from_bf16(_bf16((8, 128), 61), _bf16((8 * 64, 128), 62, 0.1).view(8, 64, 128),
                            _bf16((8 * 128, 64), 63, 0.1).view(8, 128, 64), 2)
    x, n = _bf16((20, 128), 64), w.workspace.numel()
    want = w(x).clone()
    a = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        dirty = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del dirty                                                     # the block that the next layer's workspace gets
        for _ in range(20):
            a @ a
        layer = MoETokens(w.weights.router, w.weights.w1, w.weights.w2, 2)
        got = layer(x, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        torch.cuda.synchronize()


@pytest.mark.parametrize("main_grad", [True, False])
@pytest.mark.parametrize("kw", [dict(), dict(bias=True, activation="silu")], ids=["plain", "act"])
def test_no_tokens(kw, main_grad):
    """An expert that got no token in a step: empty results and gradients, nothing added to the weight's,
    with an output gradient of any strides (sum() gives one of stride 0)."""
    log(f"no tokens {kw} main_grad={main_grad}")
    layer = _layer(64, 32, 71, fp32_main_grad=main_grad, **kw)
    if main_grad:
        layer.main_grad.fill_(2.0)
    for loss in (lambda y: y.sum(), lambda y: y.float().square().sum()):
        x = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
        y = layer(x)
        loss(y).backward()
        assert y.shape == (0, 32) and x.grad.shape == (0, 64) and layer.last_output_amax.item() == 0
        if main_grad:
            assert torch.all(layer.main_grad == 2.0)
        else:
            assert torch.count_nonzero(layer.weight.grad).item() == 0
        if layer.bias is not None:
            assert torch.count_nonzero(layer.bias_main_grad if main_grad else layer.bias.grad).item() == 0
