"""rms_norm and rms_norm_grad against 64 bits.

Bounds (u = 2^-24). A row's sum of squares: at most 16 squares after each other in a lane, 6 folds over a wave, 16
waves, all positive: 40 u relative; divided, eps added, 1/sqrt (2 u): s is within 24 u; two more products: y within
27 u < 2^-19 of its value, then one rounding to BF16 (2^-8 relative, 2^-134 below the normal numbers). dx: its two terms
within 80 u < 2^-17 of their sizes (the mean's addends 45 u of the sum of their sizes), one rounding. dw: an addend
within 27 u, and a column's addends after each other (rows of a workgroup, workgroups, 16 waves): rows + 64 additions at most."""
import numpy as np
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
import oracle
from helpers import log

pytestmark = pytest.mark.gpu
EPS = 1e-5
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _strided(g, m, n, dt, pad, std=1.0):
    return (torch.randn((m, n + pad), generator=g, device="cuda") * std).to(dt)[:, :n]


def _np(t):
    return t.double().cpu().numpy()


SHAPES = [(1, 1, 0), (3, 7, 1), (5, 31, 0), (4, 33, 3), (130, 64, 0), (9, 512, 8), (7, 513, 0), (2, 1000, 5), (600, 1032, 0), (33, 2704, 2),
          (5, 5120, 0), (1, 8192, 0), (3, 8193, 1), (2, 16384, 0), (2049, 40, 0), (70001, 40, 0),
          (31, 65, 0), (300, 100, 4), (70, 128, 0), (131, 200, 3), (35, 256, 8), (6, 257, 0)]


@pytest.mark.parametrize("m,n,pad", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(m, n, pad, dt, residual):
    log(f"rms_norm {m}x{n} pad {pad} {dt} residual {residual}")
    g = _gen(m * n)
    x = _strided(g, m, n, _DT[dt], pad)
    x[:, ::7] *= 40
    if m > 2:
        x[1] = 0                                              # a row of zeros
    r = _strided(g, m, n, _DT[dt], pad, 2.0) if residual else None
    if residual and m > 2:
        r[1] = 0
    w = (1 + 0.2 * torch.randn((n,), generator=g, device="cuda")).to(torch.bfloat16 if n % 2 else torch.float32)
    h = torch.empty_like(x) if residual else None
    q, amax = nv.FP8Tensor.empty(m, n), torch.empty((1,), device="cuda")
    y = nv.rms_norm(x, w, residual=r, eps=EPS, residual_out=h, fp8_out=q, amax_out=amax)
    torch.cuda.synchronize()
    hs = x if r is None else (x.float() + r.float()).to(x.dtype)
    if residual:
        assert torch.equal(h, hs)
    want, got = oracle.rms_norm64(_np(hs), _np(w), EPS), _np(y)
    fine = 2.0 ** -19 * np.abs(want)
    assert np.all(np.abs(got - want) <= fine + 2.0 ** -8 * (np.abs(want) + fine) + 2.0 ** -134)
    assert float(amax) == np.abs(got).max()
    # in 8 bits, from the unrounded value: the scale by its rule (up to the value's own error), every element within half a step
    s = q.scales.cpu().numpy()
    blocks = np.zeros((m, s.shape[1] * 32))
    blocks[:, :n] = np.abs(want)
    top, e = blocks.reshape(m, -1, 32).max(2), s.astype(np.int64) - 127
    assert np.all((s == 0) == (top == 0))
    on = top > 0
    assert np.all(448 * 2.0 ** e[on] >= top[on] * (1 - 2.0 ** -18))
    assert np.all((e[on] == -117) | (448 * 2.0 ** (e[on] - 1) <= top[on] * (1 + 2.0 ** -18)))
    v = oracle.fp8_dequantize(q.codes.cpu().numpy(), s)
    half = np.repeat(np.where(s == 0, 0.0, 2.0 ** (e - 10)), 32, 1)[:, :n]
    assert np.all(np.abs(v - want) <= fine + 2.0 ** -4 * np.abs(want) + half)


@pytest.mark.parametrize("m,n,pad", SHAPES)
@pytest.mark.parametrize("dt,dyt", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_gradient(m, n, pad, dt, dyt):
    log(f"rms_norm_grad {m}x{n} pad {pad} {dt} dy {dyt}")
    g = _gen(m + n)
    h, dy = _strided(g, m, n, _DT[dt], pad, 3.0), _strided(g, m, n, _DT[dyt], pad, 1e-2)
    if m > 2:
        h[2] = 0
    dr = _strided(g, m, n, _DT[dt], pad, 1e-2) if n % 3 else None
    w = 1 + 0.2 * torch.randn((n,), generator=g, device="cuda")
    dw = torch.full((n,), 0.5, device="cuda")
    add = m % 2 == 0
    dx = nv.rms_norm_grad(dy, h, w, dresidual=dr, eps=EPS, dweight=dw, accumulate=add)
    torch.cuda.synchronize()
    want, want_w, size, size_w = oracle.rms_norm_grad64(_np(dy), _np(h), _np(w), EPS, 0.0 if dr is None else _np(dr))
    fine, step = 2.0 ** -17 * size, (2.0 ** -8 if dt == "bf16" else 2.0 ** -24)
    assert np.all(np.abs(_np(dx) - want) <= fine + step * (np.abs(want) + fine) + 2.0 ** -134)
    base = 0.5 if add else 0.0
    assert np.all(np.abs(_np(dw) - (want_w + base)) <= (27 + m + 64) * 2.0 ** -24 * (size_w + base))
    # without the weight's gradient, and over its inputs
    dx2 = nv.rms_norm_grad(dy, h, w, dresidual=dr, eps=EPS, dx=None if dr is None else dr)
    torch.cuda.synchronize()
    assert torch.equal(dx2, dx)


def test_in_place_and_variants():
    g = _gen(5)
    x, r, w = _strided(g, 77, 1040, torch.bfloat16, 0), _strided(g, 77, 1040, torch.bfloat16, 0), torch.rand(1040, device="cuda")
    h, q = torch.empty_like(x), nv.FP8Tensor.empty(77, 1040)
    y = nv.rms_norm(x, w, residual=r, residual_out=h, fp8_out=q)
    for into in (x.clone(), r.clone()):
        xs, rs = (into, r) if torch.equal(into, x) else (x, into)
        y2 = nv.rms_norm(xs, w, residual=rs, residual_out=into)
        torch.cuda.synchronize()
        assert torch.equal(into, h) and torch.equal(y, y2)
    q2, amax, amax2 = nv.FP8Tensor.empty(77, 1040), torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    assert nv.rms_norm(x, w, residual=r, fp8_out=q2, fp8_only=True, amax_out=amax2) is None
    nv.rms_norm(x, w, residual=r, amax_out=amax)
    torch.cuda.synchronize()
    assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales) and torch.equal(amax, amax2)
    # no rows
    e, dw = torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda")
    assert nv.rms_norm(e, torch.ones(64, device="cuda"), amax_out=amax).shape == (0, 64) and float(amax) == 0
    nv.rms_norm_grad(e, e, torch.ones(64, device="cuda"), dweight=dw)
    assert not dw.any()


def test_values_that_are_not_finite_stay_in_their_row():
    g = _gen(6)
    x, w = _strided(g, 40, 5120, torch.bfloat16, 0), torch.rand(5120, device="cuda")
    clean, q0 = nv.rms_norm(x, w), nv.FP8Tensor.empty(40, 5120)
    nv.rms_norm(x, w, fp8_out=q0)
    x[3, 9], x[7, 5119] = float("nan"), float("inf")
    q = nv.FP8Tensor.empty(40, 5120)
    y = nv.rms_norm(x, w, fp8_out=q)
    torch.cuda.synchronize()
    rows = [i for i in range(40) if i not in (3, 7)]
    assert torch.equal(y[rows], clean[rows]) and torch.equal(q.codes[rows], q0.codes[rows])
    assert y[3].isnan().all() and y[7, 5119].isnan() and (q.scales[3] == 255).all()


def test_refusals():
    x, w = torch.randn(4, 64, device="cuda").bfloat16(), torch.ones(64, device="cuda")
    bad = nv.NVFP4Error
    with pytest.raises(bad, match="weight"):
        nv.rms_norm(x, w[:32])
    with pytest.raises(bad, match="residual"):
        nv.rms_norm(x, w, residual=x.float())
    with pytest.raises(bad, match="without a residual"):
        nv.rms_norm(x, w, residual_out=x.clone())
    with pytest.raises(bad, match="eps"):
        nv.rms_norm(x, w, eps=0.0)
    with pytest.raises(bad, match="fp8_only"):
        nv.rms_norm(x, w, fp8_only=True)
    with pytest.raises(bad, match="y8 shape"):
        nv.rms_norm(x, w, fp8_out=nv.FP8Tensor.empty(4, 32))
    with pytest.raises(bad, match="above 16384"):
        nv.rms_norm(torch.zeros(1, 16385, device="cuda"), torch.ones(16385, device="cuda"))
    with pytest.raises(bad, match="dresidual"):
        nv.rms_norm_grad(x, x, w, dresidual=x.float())
    with pytest.raises(bad, match="dweight"):
        nv.rms_norm_grad(x, x, w, dweight=torch.ones(64, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("eps", [1e-30, 1.2e-38])
def test_norm_of_zeros_with_a_tiny_eps(eps):
    x, w = torch.zeros(3, 96, device="cuda"), torch.ones(96, device="cuda")
    assert not nv.rms_norm(x, w, eps=eps).any()
    dx = nv.rms_norm_grad(x.bfloat16(), x, w, eps=eps)
    assert not dx.any()


def test_a_subnormal_eps_is_refused():
    """Its inverse root would come out infinite, and a row of zeros NaN."""
    x, w = torch.zeros(3, 96, device="cuda"), torch.ones(96, device="cuda")
    for eps in (1.17e-38, 1e-40):
        with pytest.raises(nv.NVFP4Error, match="eps"):
            nv.rms_norm(x, w, eps=eps)
        with pytest.raises(nv.NVFP4Error, match="eps"):
            nv.rms_norm_grad(x, x, w, eps=eps)
