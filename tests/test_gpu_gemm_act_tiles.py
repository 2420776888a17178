"""nvfp4_gemm_act in the tile kernel: sizes above those that the few-row kernel takes, by the library's own
rule (few_rows below), so that a limit that moves makes these tests fail instead of leaving them to the other
kernel. Bounds as in test_gpu_gemm_act.py: bit for bit the FP32 GEMM's result plus the bias for a K that is
a multiple of 64, the GEMM's bound around the 64-bit product elsewhere."""
import ctypes

import numpy as np
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
import oracle
import workloads
from helpers import assert_bytes_equal, host, log, to_device_bf16
from test_gpu_gemm_act import ACTS, U, _bf16, _check_d, _host, _operands

pytestmark = pytest.mark.gpu

# A tile is 256 x 256, one to a compute unit (256 of them). K: a multiple of 64, or brought to one.
QUARTERS = [(1000, 4089, 192), (1000, 4089, 208)]                     # 64 tiles, a quarter of a round
QUARTERS_AFTER_A_ROUND = [(4200, 4603, 64)]                           # 306 tiles: 256 and 50
SPLIT = [(2305, 2571, 256), (2305, 2571, 272), (2600, 2000, 1360)]    # 110, 88 tiles: half a round, K in two
WHOLE = [(3000, 3501, 128), (3000, 3501, 48), (170000, 5, 64)]        # 168, 665 = 512 + 153 tiles
TILES = QUARTERS + QUARTERS_AFTER_A_ROUND + SPLIT + WHOLE


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def few_rows(m, n, k):
    """Whether launch_gemm_act gives the product to the few-row kernel."""
    rule = nv.library()._ZN5nvfp417gemm_act_few_rowsElll
    rule.restype, rule.argtypes = ctypes.c_bool, [ctypes.c_int64] * 3
    return rule(m, n, k)


@pytest.mark.parametrize("mnk", TILES, ids=str)
def test_gemm_act(mnk):
    m, n, k = mnk
    log(f"gemm_act tiles {mnk}")
    assert not few_rows(m, n, k)
    if k % 64 == 0:
        assert (nv.workspace_size(nv.OP_GEMM_ACT, m, n, k) > 0) == (mnk in SPLIT)
    qa, qb = _operands(m, n, k, 1900 + m + n + k)
    if k % 64 == 0:
        d32 = _host(nv.gemm(qa, qb))
    else:
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
        what = f"gemm_act tiles {mnk} {act}"
        hb = 0.0 if bias is None else _host(bias)[None, :]
        if k % 64 == 0:
            z = (d32 + hb).astype(np.float32)
            assert_bytes_equal(_host(pre).view(np.uint32), oracle.round_bf16(z).view(np.uint32), what + " preact")
            ez = np.zeros(z.shape)
        else:
            z = d64 + hb
            ez = 1e-5 * s64 + U * np.abs(z)
            assert np.all(np.abs(_host(pre) - z) <= ez + 2.0 ** -8 * (np.abs(z) + ez) + 2.0 ** -134), what + " preact"
        _check_d(d, z, act, None if res is None else _host(res).astype(np.float64), what, ez)
        assert amax.item() == np.abs(_host(d)).max()
        if pad:                                                       # what lies between the rows stays
            for t in (out, pre):
                assert torch.count_nonzero(torch.as_strided(t, (m, n + pad), (n + pad, 1))[:, n:]).item() == 0
        assert torch.equal(nv.gemm_act(qa, qb, bias=bias, activation=act, residual=res), d), what + " alone"
        if with_res:                                                  # in place of the residual
            assert torch.equal(nv.gemm_act(qa, qb, bias=bias, activation=act, residual=res, out=res), d), what + " in place"


@pytest.mark.parametrize("mnk", [s for s in TILES if s[2] % 64 == 0], ids=str)
def test_is_the_bf16_gemm_without_extras(mnk):
    log(f"gemm_act tiles plain {mnk}")
    qa, qb = _operands(*mnk, 40)
    assert torch.equal(nv.gemm_act(qa, qb), nv.gemm_ex(qa, qb, out_dtype=torch.bfloat16))


@pytest.mark.parametrize("mnk", [QUARTERS[0], SPLIT[0], SPLIT[1], WHOLE[0]], ids=str)
def test_special_values(mnk):
    """Infinite, huge and NaN values in bias and residual stay in their columns and places, the last
    columns' and rows' too."""
    m, n, k = mnk
    log(f"gemm_act tiles special {mnk}")
    qa, qb = _operands(m, n, k, 60)
    bias = torch.zeros((n,), device="cuda")
    special = [float("inf"), float("-inf"), 3e38, -3e38, 200.0, -200.0, 40.0, -40.0]
    bias[:8] = torch.tensor(special)
    bias[n - 1] = float("inf")
    res = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    res[1, 20] = res[m - 1, n - 2] = float("nan")
    for act in ACTS:
        d = _host(nv.gemm_act(qa, qb, bias=bias, activation=act, residual=res))
        assert np.isnan(d[1, 20]) and np.isnan(d[m - 1, n - 2]) and np.isnan(d).sum() == 2, act
        assert np.all(np.isposinf(d[:, [0, n - 1]]))
        assert np.all(np.isneginf(d[:, 1]) if act == "none" else d[:, 1] == 0)
        assert np.all(np.isfinite(d[:, 4:8]))


@pytest.mark.parametrize("mnk", [QUARTERS[1], SPLIT[0], SPLIT[1], WHOLE[1]], ids=str)
def test_streams_and_graph(mnk):
    m, n, k = mnk
    log(f"gemm_act tiles graph {mnk}")
    qa, qb = _operands(m, n, k, 70)
    bias = to_device_bf16(workloads.normal_bf16((1, n), 71)).reshape(n)
    amax, amax2 = torch.zeros((1,), device="cuda"), torch.zeros((1,), device="cuda")
    want = nv.gemm_act(qa, qb, bias=bias, activation="gelu", amax_out=amax)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = nv.gemm_act(qa, qb, bias=bias, activation="gelu", stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    ws = torch.empty((nv.workspace_size(nv.OP_GEMM_ACT, m, n, k) + 256,), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.gemm_act(qa, qb, bias=bias, activation="gelu", out=out, amax_out=amax2, workspace=ws)
    for _ in range(3):
        out.fill_(7)
        amax2.fill_(1e9)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(amax, amax2)
        assert torch.equal(nv.gemm_act(qa, qb, bias=bias, activation="gelu"), want)
