"""Pins of the optimizer oracle (oracle/adamw.py) that need no GPU: the E4M3 steps against torch's
float8_e4m3fn, the scale exponent against its definition, the rounding rule's expectation, the
random bits against the generator's own words, the step against torch.optim.AdamW in float64."""
import numpy as np
import torch

import oracle
from oracle.adamw import E4M3_STEPS


def test_steps_are_e4m3():
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(E4M3_STEPS, want)


def test_scale_exponent_is_the_smallest_that_fits():
    x = np.zeros(32 * 7 + 5)
    tops = [448.0, 448.0000001, 1.0, 1.75, 1.7500001, 1e-45, 0.0, 3e38]
    x[[0, 32, 64, 96, 128, 160, 192, 224]] = tops
    x[7] = -448.0
    e = oracle.state_scale_exponents(x)
    for top, k in zip(tops, e):
        if top == 0:
            assert k == -127
        else:
            assert top <= 448 * 2.0 ** k and (k == -117 or top > 448 * 2.0 ** (k - 1))


def test_rounding_is_up_with_the_fractions_probability():
    e = np.zeros(2048, np.int64)
    h = np.arange(65536)
    for y in (0.3, 1.03, 100.1, 0.001, 447.9):
        v = oracle.state_values(oracle.state_codes(np.full(65536, y), e, h, False), e)
        gap = np.ptp(v)
        assert 0 < gap <= max(y / 8, 2.0 ** -9)
        assert -gap / 65536 <= v.mean() - y <= 1e-12                  # truncation: at most one part in 65536 low
    for y in (0.0, 1.0, 448.0, 2.0 ** -9):                           # on the grid: kept
        assert np.all(oracle.state_values(oracle.state_codes(np.full(65536, y), e, h, False), e) == y)


def test_nonzero_is_kept():
    e = np.zeros(1, np.int64)
    x = np.array([1e-9, 0.0, 1.0])
    assert list(oracle.state_codes(x, e, np.zeros(3, np.int64), True)[:2]) == [1, 0]
    assert list(oracle.state_codes(x, e, np.zeros(3, np.int64), False)[:2]) == [0, 0]
    assert oracle.state_codes(-x, e, np.zeros(3, np.int64), False)[2] == 0x80 | 0x38


def test_random_bits_are_the_generators_halves():
    h = oracle.state_random(19, tensor=3, step=7, seed=(5 << 32) | 9)
    for b in range(3):
        w = oracle.philox4x32_10(b, 0, 7, 3, 9, 5)
        for j in range(8):
            if 8 * b + j < 19:
                assert h[8 * b + j] == (int(w[j // 2]) >> (16 * (j % 2))) & 0xFFFF


def test_step_is_adamw():
    rng = np.random.default_rng(5)
    p = torch.tensor(rng.standard_normal(50), dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 4):
        g = rng.standard_normal(50)
        p.grad = torch.tensor(g)
        opt.step()
        q, m, v = oracle.adamw64(q, g, m, v, 1e-2, 0.9, 0.95, 1e-8, step, 0.1)
        assert np.allclose(p.detach().numpy(), q, rtol=1e-13, atol=1e-15)
