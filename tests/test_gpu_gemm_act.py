"""nvfp4_gemm_act and nvfp4_act_grad on the GPU.

gemm_act: the pre-activation is the FP32 GEMM's result (itself held to its bound by
test_gpu_gemm.py) plus the bias, one FP32 addition, rounded once to BF16, bit for bit. D against
act in 64 bits of that FP32 value: act's evaluation error (oracle.act_error), one FP32 addition of
the residual (u) and one rounding to BF16 (2^-8 relative, 2^-134 below the normal range). For few
rows a kernel of its own sums in another order, and for a K that is not a multiple of 64 the GEMM
itself has another kernel: there the pre-activation is held to the GEMM's bound,
ez = 1e-5 sum |a||b| + u |z| around the 64-bit product, and D to act over that range.
act_grad: dZ likewise with oracle.act_slope_error and one product (u); dbias sums M terms, each
addition within u of the running sum: (M + 2) u of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
import oracle
import workloads
from helpers import assert_bytes_equal, host, log, to_device_bf16

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACTS = ("none", "relu2", "gelu", "silu")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _host(t):
    return t.detach().float().cpu().numpy()


def _operands(m, n, k, seed):
    qa, _ = nv.quantize(to_device_bf16(workloads.with_outliers_bf16((m, k), seed)), "1x16", "rn")
    qb, _ = nv.quantize(to_device_bf16(workloads.normal_bf16((n, k), seed + 1, std=0.05)), "1x16", "rn")
    return qa, qb


def _bf16(shape, seed, std=1.0, pad=0):
    """BF16 values [rows, cols], with `pad` columns more in every row's stride."""
    rows, cols = shape
    t = torch.zeros((rows, cols + pad), dtype=torch.bfloat16, device="cuda")
    t[:, :cols] = to_device_bf16(workloads.normal_bf16(shape, seed, std=std))
    return t[:, :cols]


def _check_d(d, z32, act, res, what, ez=0.0):
    want = oracle.act64(z32, act)
    steepest = {"none": 1.0, "relu2": 2 * (np.maximum(z32, 0) + ez), "gelu": 1.13, "silu": 1.1}[act]
    tol = oracle.act_error(z32, act) + steepest * ez
    if res is not None:
        want = want + res
        tol = tol + U * np.abs(want)
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134
    err = np.abs(_host(d).astype(np.float64) - want)
    assert np.all(err <= tol), f"{what}: {(err > tol).sum()} elements, first {np.argwhere(err > tol)[0]}"


# one row; few rows on both sides of 16, 32 and 64; a K that ends inside a step of 64, 128 and 256;
# odd N (rows on any boundary); then the tile kernel: odd sizes, operands brought to a K of 128, 2752
# and 64, 90 tiles of 256 x 256 (split along K), a last round in column quarters
SHAPES = [(1, 272, 256), (1, 48, 16), (1, 1, 16), (3, 2, 16), (2, 1, 48), (1, 3, 80), (4, 70, 32), (2, 33, 80), (7, 1857, 272), (16, 512, 1344), (17, 520, 2688), (33, 256, 2704),
          (63, 100, 640), (64, 1000, 512), (65, 264, 512), (300, 520, 512), (130, 257, 272), (257, 33, 128),
          (1000, 700, 1344), (1100, 2001, 576), (2050, 1030, 80), (1003, 1857, 2704), (1500, 1400, 48),
          (2304, 2560, 256), (520, 16640, 128)]


@pytest.mark.parametrize("mnk", SHAPES)
def test_gemm_act(mnk):
    m, n, k = mnk
    log(f"gemm_act {mnk}")
    qa, qb = _operands(m, n, k, 900 + m + n + k)
    d32 = _host(nv.gemm(qa, qb))
    same_order = -(-m // 64) * -(-n // 32) > 1024 and k % 64 == 0
    if not same_order:
        ah, bh = (oracle.dequantize(*host(q)).astype(np.float64) for q in (qa, qb))
        d64, s64 = ah @ bh.T, np.abs(ah) @ np.abs(bh).T
    variants = [("none", None, False, 0), ("relu2", "bf16", False, 0), ("gelu", "fp32", True, 0),
                ("silu", "bf16", True, 8), ("none", "fp32", True, 3)]
    for i, (act, bias_dt, with_res, pad) in enumerate(variants):
        bias = None
        if bias_dt is not None:
            bias = to_device_bf16(workloads.normal_bf16((1, n), 77 + i)).reshape(n)
            bias = bias if bias_dt == "bf16" else bias.float() * 1.0001
        res = _bf16((m, n), 80 + i, pad=pad) if with_res else None
        out, pre = _bf16((m, n), 1, pad=pad), _bf16((m, n), 2, pad=pad)
        amax = torch.full((1,), -1.0, device="cuda")
        d = nv.gemm_act(qa, qb, bias=bias, activation=act, residual=res, out=out, preact=pre, amax_out=amax)
        torch.cuda.synchronize()
        what = f"gemm_act {mnk} {act}"
        if same_order:
            z32 = d32 if bias is None else (d32 + _host(bias)[None, :]).astype(np.float32)
            assert_bytes_equal(_host(pre).view(np.uint32), oracle.round_bf16(z32).view(np.uint32), what + " preact")
            ez = np.zeros(z32.shape)
        else:
            z32 = d64 + (0.0 if bias is None else _host(bias).astype(np.float64)[None, :])
            ez = 1e-5 * s64 + U * np.abs(z32)
            assert np.all(np.abs(_host(pre) - z32) <= ez + 2.0 ** -8 * (np.abs(z32) + ez) + 2.0 ** -134), what + " preact"
        _check_d(d, z32, act, None if res is None else _host(res).astype(np.float64), what, ez)
        assert amax.item() == np.abs(_host(d)).max()
        if pad:                                                       # what lies between the rows stays
            full = torch.as_strided(out, (m, n + pad), (n + pad, 1))
            assert torch.count_nonzero(full[:, n:]).item() == 0
        again = nv.gemm_act(qa, qb, bias=bias, activation=act, residual=res)
        assert torch.equal(again, d), what + " without the optional outputs"


def test_gemm_act_is_the_bf16_gemm_without_extras():
    log("gemm_act plain")
    for m, n, k in ((2000, 1300, 512), (2304, 2560, 256)):
        qa, qb = _operands(m, n, k, 40)
        assert torch.equal(nv.gemm_act(qa, qb), nv.gemm_ex(qa, qb, out_dtype=torch.bfloat16))


@pytest.mark.parametrize("m", [3, 300, 8000])
def test_residual_in_place(m):
    log(f"gemm_act residual in place {m}")
    qa, qb = _operands(m, 264, 512, 50)
    res = _bf16((m, 264), 51)
    want = nv.gemm_act(qa, qb, residual=res, activation="silu")
    got = nv.gemm_act(qa, qb, residual=res, activation="silu", out=res)
    assert torch.equal(got, want)


@pytest.mark.parametrize("m,n", [(5, 64), (260, 64), (1100, 2048)])
def test_signs_and_special_values(m, n):
    """Large and tiny pre-activations, an infinite bias, NaN in the residual: each stays in its place."""
    log(f"gemm_act special {m} {n}")
    qa, qb = _operands(m, n, 128, 60)
    bias = torch.zeros((n,), device="cuda")
    bias[:8] = torch.tensor([float("inf"), float("-inf"), 3e38, -3e38, 200.0, -200.0, 40.0, -40.0])
    res = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    res[1, 20] = float("nan")
    for act in ACTS:
        d = _host(nv.gemm_act(qa, qb, bias=bias, activation=act, residual=res))
        assert np.isnan(d[1, 20]) and np.isnan(d).sum() == 1, act
        assert np.all(np.isposinf(d[:, 0]))
        assert np.all(np.isneginf(d[:, 1]) if act == "none" else d[:, 1] == 0)
        assert np.all(np.isfinite(d[:, 4:8]))


def test_gemm_act_streams_and_graph():
    """On another stream, and in a captured graph replayed with other work between."""
    log("gemm_act graph")
    for m in (4, 300, 4100):
        qa, qb = _operands(m, 520, 512, 70)
        bias = to_device_bf16(workloads.normal_bf16((1, 520), 71)).reshape(520)
        amax, amax2 = torch.zeros((1,), device="cuda"), torch.zeros((1,), device="cuda")
        want = nv.gemm_act(qa, qb, bias=bias, activation="gelu", amax_out=amax)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        got = nv.gemm_act(qa, qb, bias=bias, activation="gelu", stream=s)
        s.synchronize()
        assert torch.equal(got, want)
        out = torch.zeros_like(want)
        ws = torch.empty((nv.workspace_size(nv.OP_GEMM_ACT, m, 520, 512) + 256,), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nv.gemm_act(qa, qb, bias=bias, activation="gelu", out=out, amax_out=amax2, workspace=ws)
        for _ in range(3):
            out.fill_(7)
            amax2.fill_(1e9)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(amax, amax2)


GRADS = [(1, 1), (1, 8), (3, 33), (8, 512), (9, 520), (123, 1857), (128, 131), (129, 131), (260, 7), (300, 1024), (2000, 72), (4100, 520)]


@pytest.mark.parametrize("mn", GRADS)
@pytest.mark.parametrize("dy32", [False, True], ids=["bf16", "fp32"])
def test_act_grad(mn, dy32):
    m, n = mn
    log(f"act_grad {mn} dy32={dy32}")
    for i, act in enumerate(ACTS):
        for pad in (0, 8, 5):
            dy = _bf16((m, n), 10 + i, pad=pad)
            if dy32:
                wide = torch.zeros((m, n + pad), device="cuda")
                wide[:, :n] = dy.float() * 1.0001
                dy = wide[:, :n]
            z = _bf16((m, n), 20 + i, std=2.0, pad=pad)
            dbias = torch.full((n,), 3.0, device="cuda")
            dz = nv.act_grad(dy, z, activation=act, dbias=dbias)
            g, zh = _host(dy).astype(np.float64), _host(z)
            want = g * oracle.act_slope64(zh, act)
            tol = np.abs(g) * (oracle.act_slope_error(zh, act) + U * np.abs(oracle.act_slope64(zh, act)))
            err = np.abs(_host(dz) - want)
            assert np.all(err <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134), f"dz {act} {mn}"
            btol = tol.sum(0) + (m + 2) * U * (np.abs(want) + tol).sum(0)
            assert np.all(np.abs(_host(dbias) - want.sum(0)) <= btol), f"dbias {act} {mn}"
            first = dbias.clone()
            dz2 = nv.act_grad(dy, z, activation=act, dbias=dbias, accumulate=True)
            assert torch.equal(dz2, dz) and torch.equal(dbias, first + first), "accumulate"
            alone = torch.empty_like(dbias)
            assert nv.act_grad(dy, z, activation=act, dbias=alone, bias_only=True) is None
            assert torch.equal(alone, first)
            assert torch.equal(nv.act_grad(dy, z, activation=act), dz)


@pytest.mark.parametrize("act", ACTS)
def test_act_grad_against_differences(act):
    """With dY = 1, dZ is the slope: against central differences of act in 64 bits (error below
    1e-9 there), within act_slope_error and the BF16 rounding."""
    log(f"act_grad differences {act}")
    z = _bf16((64, 512), 31, std=3.0)
    zh, h = _host(z).astype(np.float64), 1e-5
    diff = (oracle.act64(zh + h, act) - oracle.act64(zh - h, act)) / (2 * h)
    dz = _host(nv.act_grad(torch.ones_like(z), z, activation=act))
    tol = oracle.act_slope_error(zh, act) + 1e-8
    assert np.all(np.abs(dz - diff) <= tol + 2.0 ** -8 * (np.abs(diff) + tol) + (np.abs(zh) < 2 * h) * 2 * h)


def test_act_grad_special_values():
    log("act_grad special")
    z = torch.tensor([[float("inf"), float("-inf"), 3e38, -3e38, 100.0, -100.0, 0.0, float("nan")]],
                     dtype=torch.bfloat16, device="cuda")
    for act, want in (("gelu", [1, 0, 1, 0, 1, 0, 0.5]), ("silu", [1, 0, 1, 0, 1, 0, 0.5]),
                      ("relu2", [np.inf, 0, np.inf, 0, 200, 0, 0])):
        d = _host(nv.act_grad(torch.ones_like(z), z, activation=act))[0]
        assert np.array_equal(d[:7], np.array(want, np.float32)) or np.allclose(d[:7], want, atol=1e-30), (act, d)
        assert np.isnan(d[7])


def test_empty():
    log("gemm_act empty")
    qa, qb = _operands(4, 32, 64, 5)
    none = nv.NVFP4Tensor.empty(0, 64)
    none.global_scale.fill_(1.0)
    amax = torch.full((1,), 5.0, device="cuda")
    assert nv.gemm_act(none, qb, amax_out=amax).shape == (0, 32) and amax.item() == 0
    dbias = torch.full((32,), 3.0, device="cuda")
    e = torch.zeros((0, 32), dtype=torch.bfloat16, device="cuda")
    nv.act_grad(e, e, activation="silu", dbias=dbias, accumulate=True)
    assert torch.all(dbias == 3.0)
    assert nv.act_grad(e, e, activation="silu", dbias=dbias).shape == (0, 32) and torch.all(dbias == 0)


def test_refusals():
    qa, qb = _operands(32, 48, 64, 5)
    cuda = dict(device="cuda", dtype=torch.bfloat16)
    bad = [dict(activation="tanh"), dict(bias=torch.zeros((47,), **cuda)), dict(bias=torch.zeros((48,), device="cuda").half()),
           dict(bias=torch.zeros((96,), **cuda)[::2]), dict(residual=torch.zeros((32, 47), **cuda)),
           dict(residual=torch.zeros((32, 48), device="cuda")), dict(preact=torch.zeros((31, 48), **cuda)),
           dict(out=torch.zeros((32, 48), device="cuda")), dict(amax_out=torch.zeros((1,), **cuda)),
           dict(residual=torch.zeros((1, 48), **cuda).expand(32, 48))]
    for kw in bad:
        with pytest.raises(nv.NVFP4Error):
            nv.gemm_act(qa, qb, **kw)
    with pytest.raises(nv.NVFP4Error, match="K mismatch"):
        nv.gemm_act(qa, nv.NVFP4Tensor.empty(48, 80))
    dy, z = torch.zeros((32, 48), **cuda), torch.zeros((32, 48), **cuda)
    for args, kw in (((dy,), dict(activation="gelu")), ((dy, z[:, :40]), dict(activation="gelu")),
                     ((dy, z), dict(dbias=torch.zeros((47,), device="cuda"))), ((dy, z), dict(bias_only=True)),
                     ((dy[:1].expand(32, 48), z), dict(activation="gelu")), ((dy.half(), z), {})):
        with pytest.raises(nv.NVFP4Error):
            nv.act_grad(*args, **kw)
