"""AdamW with FP32 or 8-bit states in 64 bits (oracle; test infrastructure only), written from
the formulas stated in include/nvfp4.h at nvfp4_adamw. E4M3 values come from formats.e4m3_decode,
the random bits from philox.philox4x32_10."""
from __future__ import annotations

import numpy as np

from .formats import e4m3_decode
from .philox import philox4x32_10

E4M3_STEPS = e4m3_decode(np.arange(127, dtype=np.uint8)).astype(np.float64)   # ascending, 0 .. 448


def adamw64(p, grad, m, v, lr, beta1, beta2, eps, step, weight_decay, clip=1.0):
    """(p', m', v') in float64."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, grad, m, v))
    g = g * clip
    m2 = beta1 * m + (1 - beta1) * g
    v2 = beta2 * v + (1 - beta2) * g * g
    upd = (m2 / (1 - beta1 ** step)) / (np.sqrt(v2 / (1 - beta2 ** step)) + eps)
    return p * (1 - lr * weight_decay) - lr * upd, m2, v2


def state_scale_exponents(x):
    """Exponent e of every block of 32 (the last may be short): the smallest with max|x| <=
    448 * 2^e, at least -117; -127 where the block is zero."""
    x = np.abs(np.asarray(x, np.float64)).reshape(-1)
    x = np.concatenate([x, np.zeros(-x.size % 32)]).reshape(-1, 32).max(1)
    e = np.full(x.shape, -117, np.int64)
    for i, top in enumerate(x):
        if top == 0:
            e[i] = -127
            continue
        while top > 448 * 2.0 ** e[i]:
            e[i] += 1
    return e


def state_random(n, tensor, step, seed):
    """The 16 random bits of each of n elements of tensor number `tensor`."""
    b = np.arange((n + 7) // 8, dtype=np.uint64)
    w = philox4x32_10(b & np.uint64(0xFFFFFFFF), b >> np.uint64(32), np.uint64(step & 0xFFFFFFFF),
                      np.uint64(tensor), np.uint64(seed & 0xFFFFFFFF), np.uint64((seed >> 32) & 0xFFFFFFFF))
    words = np.stack([np.broadcast_to(x, b.shape) for x in w], 1)
    halves = np.stack([words & np.uint32(0xFFFF), words >> np.uint32(16)], 2)
    return halves.reshape(-1)[:n].astype(np.int64)


def state_codes(x, e, h, keep_nonzero):
    """Codes of x given the block exponents e and the random bits h: the E4M3 value below |x| 2^-e,
    or the next one iff fraction + h / 65536 >= 1."""
    x = np.asarray(x, np.float64).reshape(-1)
    y = np.minimum(np.abs(x) * 2.0 ** -np.repeat(e, 32)[: x.size].astype(np.float64), 448.0)
    k = np.searchsorted(E4M3_STEPS, y, side="right") - 1
    up = np.minimum(k + 1, 126)
    gap = E4M3_STEPS[up] - E4M3_STEPS[k]
    frac = np.where(gap > 0, (y - E4M3_STEPS[k]) / np.where(gap > 0, gap, 1), 0)
    k = np.where(frac + h / 65536 >= 1, up, k)
    if keep_nonzero:
        return np.where((x > 0) & (k == 0), 1, k).astype(np.uint8)
    return (k | np.where(x < 0, 128, 0)).astype(np.uint8)


def state_values(codes, e):
    """Values of codes with block exponents e."""
    codes = np.asarray(codes, np.uint8).reshape(-1)
    v = E4M3_STEPS[codes & 127] * np.where(codes > 127, -1.0, 1.0)
    s = np.where(e == -127, 0.0, 2.0 ** e.astype(np.float64))
    return v * np.repeat(s, 32)[: codes.size]
