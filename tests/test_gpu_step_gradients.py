"""What the step's modules do with gradients at the edges of their use."""
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
from bit_block_scaled_quantize_amd.moe import combine_tokens

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
