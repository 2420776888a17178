"""Outputs and workspaces that the caller gives: rows apart by any number of elements, on a stream of their own, with what lies
between the rows left as it was; bit for bit what the same call allocates by itself."""
import pytest
import torch

import bit_block_scaled_quantize_amd as nv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rand(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * std


def _apart(rows, cols, dtype, pad):
    """[rows, cols] inside rows of cols + pad elements, beginning `pad` elements into the buffer, and a check of the rest."""
    flat = torch.full((rows * (cols + pad) + pad,), 7.0, dtype=dtype, device="cuda")
    view = flat[pad:].as_strided((rows, cols), (cols + pad, 1))
    inside = torch.zeros(flat.shape, dtype=torch.bool, device="cuda")
    inside[pad:].as_strided((rows, cols), (cols + pad, 1)).fill_(True)
    return view, lambda: bool((flat[~inside] == 7.0).all())


def _same(call, outs, names):
    """call(**outs) on another stream against call() on this one."""
    want = call()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    given = {n: _apart(*o) for n, o in zip(names, outs)}
    stream.wait_stream(torch.cuda.current_stream())
    call(stream=stream, **{n: v for n, (v, _) in given.items()})
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    want = want if isinstance(want, tuple) else (want,)
    for w, (n, (view, untouched)) in zip(want, given.items()):
        assert torch.equal(view, w), n
        assert untouched(), n


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_tokens_by_expert(pad, dt):
    t, k, e, h = 90, 3, 7, 133
    s = nv.moe_sort(torch.randint(-1, e, (t, k), device="cuda", dtype=torch.int32), e)
    x, y, w = _rand(1, t, h).to(dt), _rand(2, s.rows, h).to(dt), torch.rand((t, k), device="cuda")
    _same(lambda **kw: nv.moe_gather(x, s, weights=w, **kw), [(s.rows, h, dt, pad)], ["out"])
    for out in (torch.bfloat16, torch.float32):
        _same(lambda **kw: nv.moe_combine(y, s, w, out_dtype=out, **kw), [(t, h, out, pad)], ["out"])
        dout = _rand(3, t, h).to(out)
        _same(lambda **kw: nv.moe_combine_grad(dout, y, s, w, **kw)[0], [(s.rows, h, out, pad)], ["dy"])


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("n", [100, 1040])
def test_norm(pad, n):
    m = 37
    x, r, w = _rand(1, m, n).bfloat16(), _rand(2, m, n).bfloat16(), _rand(3, n)
    _same(lambda **kw: nv.rms_norm(x, w, residual=r, **kw), [(m, n, torch.bfloat16, pad)], ["out"])
    h, untouched = _apart(m, n, torch.bfloat16, pad)
    nv.rms_norm(x, w, residual=r, residual_out=h)
    assert torch.equal(h, (x.float() + r.float()).bfloat16()) and untouched()
    _same(lambda **kw: nv.rms_norm_grad(x, r, w, **kw), [(m, n, torch.bfloat16, pad)], ["dx"])
    q = nv.fp8_quantize(x)
    _same(lambda **kw: nv.fp8_dequantize(q, **kw), [(m, n, torch.bfloat16, pad)], ["out"])


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("t,h,v", [(20, 48, 333), (150, 112, 333), (300, 528, 2100)])
def test_head(pad, t, h, v):
    x, w = _rand(1, t, h).bfloat16(), _rand(2, v, h, std=0.1).bfloat16()
    tg, gr = torch.randint(-5, v, (t,), device="cuda"), torch.rand(t, device="cuda")
    loss, lse = nv.linear_cross_entropy(x, w, tg)
    names = ["dx", "dweight"]
    grad = lambda **kw: nv.linear_cross_entropy_grad(x, w, tg, lse, gr, loss=loss, **kw)  # noqa: E731
    _same(grad, [(t, h, torch.bfloat16, pad), (v, h, torch.bfloat16, pad)], names)
    d32, untouched = _apart(v, h, torch.float32, pad)
    base = _rand(5, v, h)
    d32.copy_(base)
    grad(dweight=d32, accumulate=True)
    alone = torch.zeros((v, h), device="cuda")
    grad(dweight=alone, accumulate=True)
    assert torch.equal(d32, base + alone) and untouched()
    # a workspace of the caller's, larger than needed and full of NaN, and given buffers for the losses
    for op, call in ((nv.OP_HEAD_LOSS, lambda ws: nv.linear_cross_entropy(x, w, tg, loss=torch.empty_like(loss), lse=torch.empty_like(lse), workspace=ws)),
                     (nv.OP_HEAD_GRAD, lambda ws: grad(workspace=ws))):
        ws = torch.full((nv.workspace_size(op, t, v, h) + 512,), 0xFF, dtype=torch.uint8, device="cuda")
        for a, b in zip(call(ws), call(None)):
            assert torch.equal(a, b)
        assert bool((ws[-512:] == 0xFF).all())
