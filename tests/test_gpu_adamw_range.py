"""Where nvfp4_adamw's squares leave FP32, as include/nvfp4.h states it."""
import numpy as np
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
import oracle
from helpers import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _tensor(g):
    z = lambda v: torch.full((len(g),), v, device="cuda")  # noqa: E731
    return nv.AdamWTensor(p=z(1.0), grad=torch.tensor(g, dtype=torch.float32, device="cuda"), m=z(0.0), v=z(0.0))


@pytest.mark.parametrize("size,count,finite", [(1.8e19, 1, True), (1.9e19, 1, False), (6.4e18, 8, True), (6.6e18, 8, False),
                                               (3e-23, 1, True), (2e-23, 8, True)])
def test_norm(size, count, finite):
    """count equal gradients next to each other among zeros."""
    log(f"adamw norm of {count} x {size}")
    g = np.zeros(4096)
    g[2056:2056 + count] = size
    t = _tensor(g)
    norm = nv.adamw(nv.AdamWPlan([t]), lr=1e-2, step=1, max_norm=1.0).item()
    p = t.p.cpu().numpy().astype(np.float64)
    if not finite:
        assert np.isinf(norm) and np.all(p == 1)
        return
    true = size * np.sqrt(count)
    if size == 2e-23:
        assert norm == 0                                              # their squares are below FP32
    elif size == 3e-23:
        assert 0 < norm <= 2 * true                                   # the square has one bit
    else:
        assert abs(norm - true) <= 20 * U * true
        clip = 1.0 / (true + 1e-6)
        want, _, _ = oracle.adamw64(np.ones(4096), np.float32(g), np.zeros(4096), np.zeros(4096), 1e-2, 0.9, 0.95, 1e-8, 1, 0.0, clip)
        assert np.all(np.abs(p - want) <= 1e-2 * 40 * U + 4 * U)      # an update of lr, 40 roundings; p's own


def test_small_r_in_8_bits():
    """With no gradient an r of 2^-74 goes on, one of 2^-76 ends; m and p move by nothing that counts."""
    log("adamw small r")
    r = np.repeat([2.0 ** -74, 2.0 ** -76], 32)
    e = oracle.state_scale_exponents(r)
    z = lambda: torch.zeros((64,), dtype=torch.uint8, device="cuda")  # noqa: E731
    v = torch.from_numpy(oracle.state_codes(r, e, np.full(64, 32768), True)).cuda()
    t = nv.AdamWTensor(p=torch.ones(64, device="cuda"), grad=torch.zeros(64, device="cuda"), m=z(), v=v, m_scale=z()[:2],
                       v_scale=torch.from_numpy((e + 127).astype(np.uint8)).cuda())
    nv.adamw(nv.AdamWPlan([t]), lr=1e-2, step=2)
    got = oracle.state_values(t.v.cpu().numpy(), t.v_scale.cpu().numpy().astype(np.int64) - 127)
    assert np.all(got[:32] > 2.0 ** -75) and np.all(got[32:] == 0)
    assert torch.all(t.p == 1)
