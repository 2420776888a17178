"""What the step's modules do with gradients at the edges of their use: types that differ between the two sides, second
derivatives, 8-bit tensors of other shapes, tables that end below the rows, a captured
step of the head."""
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


def test_weight_gradients_by_expert_with_rows_behind_the_last():
    """rht_quantize with the sort's offsets as segments and grouped_gemm_k over them, the offsets ending below the rows: each expert's
    gradient is that of its own rows."""
    t, k, e, h, n = 200, 2, 5, 128, 96
    rng = torch.Generator().manual_seed(7)
    ids = torch.randint(-1, e - 1, (t, k), generator=rng, dtype=torch.int32).cuda()     # the last expert gets none
    s = nv.moe_sort(ids, e)
    off = s.offsets.tolist()
    assert off[-1] < s.rows and off[-1] == off[-2]
    x, dy = nv.moe_gather(_rand(1, t, h).bfloat16(), s), nv.moe_gather(_rand(2, t, n).bfloat16(), s)
    a, b = (nv.rht_quantize(m, 0x1234, segments=s.offsets) for m in (dy, x))
    d = nv.grouped_gemm_k(s.offsets, a, b)
    for g in range(e):
        lo, hi = off[g], off[g + 1]
        got = d[g * n:(g + 1) * n]
        if lo == hi:
            assert not got.any()
            continue
        one, two = (nv.rht_quantize(m[lo:hi].contiguous(), 0x1234) for m in (dy, x))
        assert torch.equal(one.global_scale, a.global_scale[g:g + 1]) and torch.equal(two.global_scale, b.global_scale[g:g + 1])
        assert torch.equal(one.codes, a.codes[:, lo // 2:hi // 2]) and torch.equal(two.scales, b.scales[:, lo // 16:hi // 16])
        ref = nv.dequantize(one).double() @ nv.dequantize(two).double().t()
        size = nv.dequantize(one).double().abs() @ nv.dequantize(two).double().abs().t()
        assert bool(((got.double() - ref).abs() <= 1e-5 * size).all())


@pytest.mark.parametrize("block", ["1x16", "16x16"])
@pytest.mark.parametrize("last", [0, 64])
def test_rows_behind_the_last_segment_count_as_its(block, last):
    """A table that ends below the rows gives what the same table gives with the rows as its end, in quantize, rht_quantize and amax."""
    rows, cols = 320, 96
    x = _rand(1, rows, cols).bfloat16()
    x[200:] *= 3
    short = torch.tensor([0, 64, 128, 128 + last], device="cuda")
    whole = torch.tensor([0, 64, 128, rows], device="cuda")
    for call in (lambda s: nv.quantize(x, block, segments=s)[0], lambda s: nv.rht_quantize(x, 0x77, segments=s)):
        a, b = call(short), call(whole)
        for one, two in ((a.codes, b.codes), (a.scales, b.scales), (a.global_scale, b.global_scale)):
            assert torch.equal(one, two)
    for rht in (False, True):
        assert torch.equal(nv.amax(x, segments=short, rht=rht), nv.amax(x, segments=whole, rht=rht))


@pytest.mark.parametrize("reduction", ["mean", "sum"])
@pytest.mark.parametrize("t", [300, 40000])
def test_captured_step_of_the_head(reduction, t):
    """Forward and backward of the module in one graph, replayed several times with other work between; each is the eager result."""
    h, v = 32, 130
    head = LinearCrossEntropy(h, v, device="cuda", reduction=reduction)
    head.weight.data.copy_(_rand(1, v, h, std=0.2))
    x = _rand(2, t, h).bfloat16().requires_grad_()
    tg = torch.randint(0, v, (t,), device="cuda")

    def step():
        head.main_grad.zero_()
        loss = head(x, tg)
        dx, = torch.autograd.grad(loss, x)
        return loss.detach(), dx, head.main_grad             # nothing holds the autograd graph
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for turn in range(5):
        with torch.no_grad():
            x.copy_(_rand(10 + turn, t, h))
            tg.copy_(torch.randint(-20, v, (t,), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.detach().clone() for o in out]
        want = [o.detach().clone() for o in step()]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), turn
        torch.empty(1 << 20, device="cuda").fill_(float(turn)).sum()
