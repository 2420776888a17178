"""moe_sort, moe_gather, moe_combine and moe_combine_grad. The order is the oracle's; rows that are copied, weighted
(one FP32 product, one rounding) or added in the order of the pairs (FP32, each step rounded) are compared bit for bit
with the same steps in torch; dweights, whose products are added per lane and then over the wave, within
hidden / 64 + 16 roundings (2^-24) of the sum of their sizes."""
import numpy as np
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
import oracle
from helpers import log

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ids(t, k, e, seed, kind="mixed"):
    rng = np.random.default_rng(seed)
    if kind == "one":
        ids = np.full((t, k), e - 1)
    elif kind == "none":
        ids = np.full((t, k), -1)
    else:
        ids = np.minimum(rng.geometric(3.0 / (e + 2), (t, k)) - 1, e - 1)
        if kind == "mixed":
            ids[rng.random((t, k)) < 0.1] = -1
            ids[rng.random((t, k)) < 0.05] = e               # and past the end
    return torch.from_numpy(ids.astype(np.int32)).cuda()


CASES = [(1, 1, 1, 1), (1, 8, 8, 64), (7, 3, 24, 64), (64, 2, 5, 16), (341, 3, 128, 64), (342, 3, 128, 1), (1000, 6, 128, 64), (513, 2, 1024, 64),
         (3000, 8, 3, 64), (5000, 1, 300, 128), (9, 7, 1000, 3)]


@pytest.mark.parametrize("t,k,e,align", CASES)
@pytest.mark.parametrize("kind", ["mixed", "full", "one", "none"])
def test_order(t, k, e, align, kind):
    log(f"moe_sort {t}x{k} of {e}, align {align}, {kind}")
    ids = _ids(t, k, e, t + e, kind)
    s = nv.moe_sort(ids, e, align)
    offsets, row_of, pair_of = oracle.moe_order(ids.cpu().numpy(), e, align, s.rows)
    np.testing.assert_array_equal(s.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(s.row_of.cpu().numpy(), row_of)
    np.testing.assert_array_equal(s.pair_of.cpu().numpy(), pair_of)


def test_order_of_many():
    """More chunks than one share of the scan takes at a time, against a stable sort."""
    t, k, e = 200000, 8, 7
    ids = _ids(t, k, e, 1, "full")
    s = nv.moe_sort(ids, e, 64)
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(s.pair_of[s.pair_of >= 0].long(), order)
    count = torch.bincount(flat, minlength=e)
    assert torch.equal(s.offsets[1:], ((count + 63) // 64 * 64).cumsum(0))
    rows = s.row_of.reshape(-1).long()
    assert torch.equal(s.pair_of[rows].long(), torch.arange(t * k, device="cuda"))


def test_nothing():
    s = nv.moe_sort(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 6, 64)
    assert s.rows == 0 and not s.offsets.any() and s.offsets.numel() == 7
    x = torch.empty((0, 32), device="cuda")
    assert nv.moe_gather(x, s).shape == (0, 32) and nv.moe_combine(x, s).shape == (0, 32)
    dy, dw = nv.moe_combine_grad(x, x, s, torch.empty((0, 4), device="cuda"))
    assert dy.shape == (0, 32) and dw.shape == (0, 4)


@pytest.mark.parametrize("pairs,e", [(512 * 4096, 40), (512 * 4096 + 1, 40), (2300001, 1024)])
def test_order_by_a_launch_between(pairs, e):
    """Around the number of chunks from which the counts are added up in a launch of its own."""
    log(f"moe_sort {pairs} pairs of {e}")
    ids = torch.from_numpy(np.random.default_rng(pairs).integers(-1, e + 1, pairs).astype(np.int32)).cuda()
    s = nv.moe_sort(ids.view(-1, 1), e, 64)
    flat, p = ids.long(), torch.arange(pairs, device="cuda")
    valid = (flat >= 0) & (flat < e)
    order = torch.sort(torch.where(valid, flat, e), stable=True).indices[:int(valid.sum())]
    assert torch.equal(s.pair_of[s.pair_of >= 0].long(), order)
    count = torch.bincount(flat[valid], minlength=e)
    assert s.offsets[0] == 0 and torch.equal(s.offsets[1:], ((count + 63) // 64 * 64).cumsum(0))
    rows = s.row_of.reshape(-1).long()
    assert torch.equal(rows >= 0, valid) and torch.equal(s.pair_of[rows[valid]].long(), p[valid])
    first = s.offsets[flat[valid]]
    assert bool(((rows[valid] >= first) & (rows[valid] < first + count[flat[valid]])).all())


@pytest.mark.parametrize("t,k,e,align", [c for c in CASES if c[0] < 4000])
@pytest.mark.parametrize("h,pad", [(1, 0), (37, 3), (512, 0), (1040, 8)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows(t, k, e, align, h, pad, dt):
    log(f"gather, combine {t}x{k} of {e}, hidden {h}+{pad} {dt}")
    g = torch.Generator(device="cuda")
    g.manual_seed(t * h)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    ids = _ids(t, k, e, t + e)
    s = nv.moe_sort(ids, e, align)
    has, at = s.pair_of >= 0, s.pair_of.clamp_min(0).long()
    x, w = rand(t, h + pad).to(dt)[:, :h], torch.rand((t, k), generator=g, device="cuda")
    w[s.row_of < 0] = float("nan")                            # weights of dropped pairs are not looked at
    zero = torch.zeros((), dtype=dt, device="cuda")
    got = nv.moe_gather(x, s)
    assert torch.equal(got, torch.where(has[:, None], x[at // k], zero))
    wr = w.reshape(-1)[at]
    got = nv.moe_gather(x, s, weights=w)
    scaled = torch.where(has[:, None], (x[at // k].float() * wr[:, None]).to(dt), zero)
    assert torch.equal(got, scaled)
    # back
    y = rand(s.rows, h + pad).to(dt)[:, :h]
    y[~has] = float("inf")                                    # rows without a pair are not read
    dout = rand(t, h + pad).bfloat16()[:, :h]
    row, on = s.row_of.clamp_min(0).long(), s.row_of >= 0
    for out_dtype in (torch.bfloat16, torch.float32):
        for weights in (None, w):
            want = torch.zeros((t, h), device="cuda")
            for j in range(k):
                term = y[row[:, j]].float()
                if weights is not None:
                    term = weights[:, j:j + 1] * term
                want = torch.where(on[:, j:j + 1], want + term, want)
            got = nv.moe_combine(y, s, weights, out_dtype=out_dtype)
            assert torch.equal(got, want.to(out_dtype))
    dy, dw = nv.moe_combine_grad(dout, y, s, w)
    want = torch.where(has[:, None], (dout[at // k].float() * wr[:, None]).bfloat16(), torch.zeros((), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(dy, want)
    yr = torch.where(on[:, :, None], y[row].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    terms = yr * dout.double()[:, None, :]
    assert bool(((dw.double() - terms.sum(2)).abs() <= (h / 64 + 16) * 2.0 ** -24 * terms.abs().sum(2)).all())
    only_y, none = nv.moe_combine_grad(dout, None, s, w, need_dweights=False)
    assert none is None and torch.equal(only_y, dy)
    none, only_w = nv.moe_combine_grad(dout, y, s, w, need_dy=False)
    assert none is None and torch.equal(only_w, dw)


def test_grouped_products_take_the_order():
    """quantize with the offsets as segments and grouped_gemm over the padded rows: the rows behind the last
    expert's belong to no product, and each expert's rows are its plain product's."""
    t, k, e, h, n = 200, 2, 5, 128, 96
    ids = _ids(t, k, e, 3)
    s = nv.moe_sort(ids, e, 64)
    x = torch.randn(t, h, device="cuda").bfloat16()
    xs = nv.moe_gather(x, s)
    w = torch.randn(e * n, h, device="cuda").bfloat16()
    seg = torch.arange(e + 1, dtype=torch.int64, device="cuda") * n
    qx, _ = nv.quantize(xs, segments=s.offsets)
    qw, _ = nv.quantize(w, "16x16", segments=seg)
    d = torch.full((s.rows, n), 7.0, device="cuda")
    nv.grouped_gemm(s.offsets, qx, qw, n, out=d)
    off = s.offsets.tolist()
    assert off[-1] < s.rows and (d[off[-1]:] == 7.0).all()
    for g in range(e):
        a, b = off[g], off[g + 1]
        if a == b:
            continue
        one, _ = nv.quantize(xs[a:b].contiguous())
        we, _ = nv.quantize(w[g * n:(g + 1) * n].contiguous(), "16x16")
        assert torch.equal(nv.dequantize(one), nv.dequantize(nv.NVFP4Tensor(qx.codes[a:b].contiguous(), qx.scales[a:b].contiguous(),
                                                                             qx.global_scale[g:g + 1].contiguous(), b - a, h)))
        ref = nv.dequantize(one).double() @ nv.dequantize(we).double().t()
        size = nv.dequantize(one).double().abs() @ nv.dequantize(we).double().abs().t()
        assert bool(((d[a:b].double() - ref).abs() <= 1e-5 * size).all())


def test_tables_that_are_wrong_do_no_harm():
    """row_of and pair_of are device data: what is out of range counts as no row, no pair."""
    s = nv.moe_sort(_ids(20, 2, 4, 1), 4, 16)
    x = torch.randn(20, 64, device="cuda")
    wild = torch.tensor([-5, 40, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    s.pair_of[:4] = wild
    xs = nv.moe_gather(x, s)
    assert not xs[:4].any()
    y = torch.randn(s.rows, 64, device="cuda")
    s.row_of[:2] = torch.tensor([[s.rows, -7], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    out = nv.moe_combine(y, s, torch.ones(20, 2, device="cuda"), out_dtype=torch.float32)
    assert not out[:2].any()
    dy, dw = nv.moe_combine_grad(x, y, s, torch.ones(20, 2, device="cuda"))
    torch.cuda.synchronize()
    assert not dw[:2].any() and not dy[:4].any()


def test_refusals():
    bad = nv.NVFP4Error
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(bad, match="ids"):
        nv.moe_sort(ids.long(), 4)
    with pytest.raises(bad, match="at most 1024"):
        nv.moe_sort(ids, 1025)
    with pytest.raises(bad, match="no sorted order"):
        nv.moe_sort(ids, 4, align=0)
    s = nv.moe_sort(ids, 4)
    x = torch.randn(4, 32, device="cuda")
    with pytest.raises(bad, match="tokens"):
        nv.moe_gather(x[:3], s)
    with pytest.raises(bad, match="out shape"):
        nv.moe_gather(x, s, out=x.clone())
    with pytest.raises(bad, match="rows"):
        nv.moe_combine(x, s)
    y = torch.randn(s.rows, 32, device="cuda")
    with pytest.raises(bad, match="weights"):
        nv.moe_combine(y, s, torch.ones(4, 2, device="cuda").double())
    with pytest.raises(bad, match="needs y"):
        nv.moe_combine_grad(x, None, s, torch.ones(4, 2, device="cuda"))
    with pytest.raises(bad, match="row_of"):
        nv.moe_combine(y, nv.MoESort(s.offsets, s.row_of[:2], s.pair_of, 4, 2))


@pytest.mark.parametrize("t,k,h,dt", [(20000, 6, 1203, torch.bfloat16), (30001, 4, 601, torch.float32), (300000, 4, 2048, torch.bfloat16)])
def test_rows_of_many(t, k, h, dt):
    """Outputs larger than the caches, one past 4 GiB; the way back, and its gradient."""
    log(f"gather, combine {t}x{k} hidden {h} {dt}")
    ids = _ids(t, k, 48, t)
    s = nv.moe_sort(ids, 48)
    g = torch.Generator(device="cuda")
    g.manual_seed(t)
    x = torch.randn((t, h), generator=g, device="cuda").to(dt)
    w = torch.randint(1, 5, (t, k), generator=g, device="cuda") / 4.0
    y, wy = nv.moe_gather(x, s), nv.moe_gather(x, s, weights=w)
    dy, dw = nv.moe_combine_grad(x, y, s, w)
    for r in range(0, s.rows, 65536):
        pair = s.pair_of[r:r + 65536].long()
        want = torch.where((pair >= 0)[:, None], x[pair.clamp_min(0) // k], torch.zeros((), dtype=dt, device="cuda"))
        assert torch.equal(y[r:r + 65536], want)
        want = (want.float() * w.reshape(-1)[pair.clamp_min(0)][:, None]).to(dt)
        assert torch.equal(wy[r:r + 65536], want) and torch.equal(dy[r:r + 65536], want)
    out = nv.moe_combine(y, s, w, out_dtype=torch.float32)
    total = torch.zeros((t,), device="cuda")                  # of the weights, multiples of a quarter: exact
    for j in range(k):
        total += torch.where(s.row_of[:, j] >= 0, w[:, j], 0.0)
    xf = x.double()
    assert bool(((out.double() - xf * total[:, None]).abs() <= k * 2.0 ** -23 * k * xf.abs()).all())
    square = xf.square().sum(1)[:, None].expand(t, k)
    bound = (h / 64 + 16) * 2.0 ** -24 * square
    assert bool(((dw.double() - torch.where(s.row_of >= 0, square, 0.0)).abs() <= bound).all())


@pytest.mark.parametrize("e,align", [(1, 2 ** 31 - 1), (2, 2 ** 30 - 1)])
def test_runs_that_end_at_the_last_row_there_is(e, align):
    """Rows up to 2^31 - 1: a count and its alignment together, and a row and the next one of its lane, are more."""
    log(f"moe_sort of {e}, align {align}")
    ids = torch.tensor([[e - 1], [0], [-1], [e - 1]], dtype=torch.int32, device="cuda")
    s = nv.moe_sort(ids, e, align)
    want = {1: ([0, align], [0, 1, -1, 2], {0: 0, 1: 1, 2: 3}), 2: ([0, align, 2 * align], [align, 0, -1, align + 1], {0: 1, align: 0, align + 1: 3})}[e]
    assert s.offsets.tolist() == want[0] and s.rows == want[0][-1] and s.row_of.reshape(-1).tolist() == want[1]
    for row, pair in want[2].items():
        assert int(s.pair_of[row]) == pair
        s.pair_of[row] = -1
    assert int(s.pair_of.min()) == int(s.pair_of.max()) == -1
