"""What the step's modules do with gradients at the edges of their use: types that differ between the two sides, second
derivatives, 8-bit tensors of other shapes."""
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
from bit_block_scaled_quantize_amd.linear import NVFP4Linear
from bit_block_scaled_quantize_amd.loss import LinearCrossEntropy
from bit_block_scaled_quantize_amd.moe import combine_tokens, gather_tokens
from bit_block_scaled_quantize_amd.norm import RMSNorm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rand(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * std


@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_combine_gradient_in_the_rows_type(y_dtype, out_dtype):
    """w dout rounded once, to y's type, whatever the output's type: FP32 products as they are, or their BF16 rounding."""
    t, k, e, h = 70, 3, 6, 264
    ids = torch.randint(-1, e, (t, k), device="cuda", dtype=torch.int32)
    s = nv.moe_sort(ids, e)
    y = _rand(1, s.rows, h).to(y_dtype).requires_grad_()
    w = torch.rand((t, k), device="cuda", requires_grad=True)
    out = combine_tokens(y, s, w, out_dtype=out_dtype)
    dout = _rand(2, t, h).to(out_dtype)
    out.backward(dout)
    has, pair = s.pair_of >= 0, s.pair_of.clamp_min(0).long()
    want = (w.detach().reshape(-1)[pair][:, None] * dout.float()[pair // k]).to(y_dtype)
    want = torch.where(has[:, None], want, torch.zeros((), dtype=y_dtype, device="cuda"))
    assert y.grad.dtype == y_dtype and torch.equal(y.grad, want)
    rows, on = s.row_of.clamp_min(0).long(), (s.row_of >= 0)
    terms = torch.where(on[:, :, None], y.detach().double()[rows], 0.0) * dout.double()[:, None, :]
    assert bool(((w.grad.double() - terms.sum(2)).abs() <= (h / 64 + 16) * 2.0 ** -24 * terms.abs().sum(2)).all())


def _second(make):
    """The gradient of `make()`'s output with respect to its leaf, as a graph, and a penalty on it."""
    out, leaf = make()
    first, = torch.autograd.grad(out.float().sum(), leaf, create_graph=True)
    return first, first.float().square().sum()


def _norm():
    x = _rand(1, 16, 64).bfloat16().requires_grad_()
    return RMSNorm(64, device="cuda")(x), x


def _head():
    x = _rand(1, 16, 64).bfloat16().requires_grad_()
    head = LinearCrossEntropy(64, 100, device="cuda")
    head.weight.data.copy_(_rand(2, 100, 64))
    return head(x, torch.arange(16, device="cuda")), x


def _gather():
    x = _rand(1, 16, 64).requires_grad_()
    return gather_tokens(x, nv.moe_sort(torch.zeros((16, 1), dtype=torch.int32, device="cuda"), 2)), x


def _combine():
    s = nv.moe_sort(torch.zeros((16, 1), dtype=torch.int32, device="cuda"), 2)
    w = torch.rand((16, 1), device="cuda", requires_grad=True)
    return combine_tokens(_rand(1, s.rows, 64), s, w), w


def _linear(**kw):
    def make():
        x = _rand(1, 16, 64).bfloat16().requires_grad_()
        layer = NVFP4Linear(64, 96, device="cuda", **kw)
        layer.weight.data.copy_(_rand(3, 96, 64, std=0.1))
        return layer(x), x
    return make


MAKERS = {"norm": _norm, "head": _head, "gather": _gather, "combine": _combine, "linear": _linear(),
          "linear with activation": _linear(activation="silu", bias=True)}


@pytest.mark.parametrize("name", MAKERS)
def test_second_derivatives_are_refused(name):
    """A penalty on a gradient raises when it is differentiated, instead of adding nothing; a gradient kept as a graph and not
    differentiated further is the ordinary one."""
    first, penalty = _second(MAKERS[name])
    out, leaf = MAKERS[name]()
    if name != "combine":                                     # its weights differ from call to call
        plain, = torch.autograd.grad(out.float().sum(), leaf)
        assert torch.equal(first, plain)
    with pytest.raises(RuntimeError, match="second"):
        penalty.backward()


def test_fp8_input_with_codes_of_another_shape():
    """x_fp8 is what its rows and columns say, however the codes' tensor is shaped, as in the other calls that take one."""
    x = _rand(1, 32, 64).bfloat16().requires_grad_()
    dy = _rand(2, 32, 96).bfloat16()
    q = nv.fp8_quantize(x.detach())
    got = []
    for codes, scales in ((q.codes, q.scales), (q.codes.reshape(-1), q.scales.reshape(-1)), (q.codes.view(2, 16, 64), q.scales.view(4, 16))):
        layer = NVFP4Linear(64, 96, device="cuda", checkpoint="fp8")
        layer.weight.data.copy_(_rand(3, 96, 64, std=0.1))
        x.grad = None
        layer(x, x_fp8=nv.FP8Tensor(codes, scales, 32, 64)).backward(dy)
        got.append((x.grad.clone(), layer.main_grad.clone()))
    for dx, dw in got[1:]:
        assert torch.equal(dx, got[0][0]) and torch.equal(dw, got[0][1])


def test_fp8_input_is_checked_before_the_forward():
    layer = NVFP4Linear(64, 96, device="cuda", checkpoint="fp8")
    torch.nn.init.normal_(layer.weight, std=0.1)
    x = _rand(1, 32, 64).bfloat16().requires_grad_()
    q = nv.fp8_quantize(x.detach())
    for codes, scales in ((q.codes[:16], q.scales), (q.codes, q.scales[:16]), (q.codes.int(), q.scales), (q.codes.cpu(), q.scales)):
        with pytest.raises(nv.NVFP4Error, match="x_fp8"):
            layer(x, x_fp8=nv.FP8Tensor(codes, scales, 32, 64))
    assert layer._calls == 0


@pytest.mark.parametrize("kw", [dict(), dict(bias=True, activation="gelu")], ids=["plain", "act"])
def test_frozen_layer_with_8_bit_checkpoints(kw):
    """The input's gradient is the trained layer's, also from no tokens; x_fp8 is not needed and does no harm."""
    x, dy = _rand(1, 32, 64).bfloat16().requires_grad_(), _rand(2, 32, 96).bfloat16()
    layer = NVFP4Linear(64, 96, device="cuda", checkpoint="fp8", **kw)
    layer.weight.data.copy_(_rand(3, 96, 64, std=0.1))
    got = []
    for frozen, q in ((False, None), (True, None), (True, nv.fp8_quantize(x.detach()))):
        layer.weight.requires_grad_(not frozen)
        layer._calls, x.grad = 0, None
        layer(x, x_fp8=q).backward(dy)
        got.append(x.grad.clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    x.grad = None
    layer(x[:0]).sum().backward()
    assert not x.grad.any()
