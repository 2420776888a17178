"""A mixture-of-experts layer in 64 bits with how far an implementation that keeps to the stated
roundings may be from it (oracle; test infrastructure only). Rules as include/nvfp4.h states them at
nvfp4_moe_tokens; the routing is an argument, so that a test can hold the routing and the
experts' products apart.

Tolerance of y: the up product is a GEMM (1e-5 sum |w||x|), the activation adds its own error
(activation.act_error), h takes one rounding to 11 significant bits (2^-11) and 2^-39 of its largest
value, the down product is a GEMM again, the routing weight one product (u) per expert, their sum k
additions (k u), the result one rounding to BF16 (2^-8)."""
from __future__ import annotations

import numpy as np

from .activation import U, act64, act_error, act_slope64


def _steepest(z, ez, act):
    if act == "relu2":
        return act_slope64(z + ez, act)
    return {"none": 1.0, "gelu": 1.13, "silu": 1.1}[act]


def moe64(x, ids, weights, w1, w2, act, gated):
    """x [T, H]; ids, weights [T, k]; w1 [E, F or 2F, H]; w2 [E, H, F], all dequantized. Returns
    (y [T, H], tolerance [T, H])."""
    x = np.asarray(x, np.float64)
    y, tol = np.zeros(x.shape), np.zeros(x.shape)
    mag = np.zeros(x.shape)
    for t in range(x.shape[0]):
        for e, w in zip(ids[t], np.asarray(weights[t], np.float64)):
            a, b = np.asarray(w1[e], np.float64), np.asarray(w2[e], np.float64)
            z = a @ x[t]
            ez = 1e-5 * (np.abs(a) @ np.abs(x[t]))
            f = z.size // 2 if gated else z.size
            h = act64(z[:f], act)
            eh = _steepest(z[:f], ez[:f], act) * ez[:f] + act_error(z[:f], act)
            if gated:
                u, eu = z[f:], ez[f:]
                eh = eh * (np.abs(u) + eu) + np.abs(h) * eu + U * np.abs(h * u)
                h = h * u
            eh = eh + 2.0 ** -11 * (np.abs(h) + eh) + 2.0 ** -39 * np.abs(h).max(initial=0)
            part = b @ h
            big = np.abs(b) @ (np.abs(h) + eh)
            y[t] += w * part
            tol[t] += abs(w) * (np.abs(b) @ eh + 1e-5 * big + 2 * U * np.abs(part))
            mag[t] += abs(w) * np.abs(part)
    tol += ids.shape[1] * U * (mag + tol)
    return y, tol + 2.0 ** -8 * (np.abs(y) + tol) + 2.0 ** -134
