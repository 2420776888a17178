"""The element functions of nvfp4_gemm_act / nvfp4_act_grad in 64 bits, and how far an FP32
evaluation may be from them (oracle; test infrastructure only). Formulas as include/nvfp4.h states
them at nvfp4_act."""
from __future__ import annotations

import numpy as np

KINDS = ("none", "relu2", "gelu", "silu")
_C = np.sqrt(2 / np.pi)
U = 2.0 ** -24


def _sigmoid(t):
    """1 / (1 + exp(-t)): (1 + tanh u) / 2 = sigmoid(2u) and 1 - sigmoid(t) = sigmoid(-t), which keep
    their relative accuracy where 1 + tanh u and 1 - s cancel."""
    return 1 / (1 + np.exp(-np.clip(t, -745, 745)))


def act64(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "relu2":
        return np.square(np.maximum(z, 0))
    if kind == "gelu":
        return z * _sigmoid(2 * _C * (z + 0.044715 * z ** 3))
    if kind == "silu":
        return z / (1 + np.exp(-z))
    return z


def act_slope64(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "relu2":
        return 2 * np.maximum(z, 0)
    if kind == "gelu":
        t = 2 * _C * (z + 0.044715 * z ** 3)
        return _sigmoid(t) * (1 + z * _sigmoid(-t) * 2 * _C * (1 + 3 * 0.044715 * z * z))
    if kind == "silu":
        return _sigmoid(z) * (1 + z * _sigmoid(-z))
    return np.ones_like(z)


def _sigmoid_parts(z, kind):
    t = z if kind == "silu" else 2 * _C * (z + 0.044715 * z ** 3)
    dt = np.ones_like(z) if kind == "silu" else 2 * _C * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + np.exp(-np.clip(t, -700, 700)))
    # t: four roundings, the exponent's base change two more on it, the exponential two units:
    # exp(-t) is within (6 |t| + 2) u, 1 / (1 + exp) within s (1 - s) of that and four more roundings
    return t, dt, s, s * (6 * np.abs(t) + 8) * U


def act_error(z, kind):
    """Bound on |FP32 evaluation - act64| at an exactly known FP32 z."""
    z = np.asarray(z, np.float64)
    if kind == "none":
        return np.zeros_like(z)
    if kind == "relu2":
        return 2 * U * act64(z, kind)
    _, _, s, ds = _sigmoid_parts(z, kind)
    return np.abs(z) * (ds + 2 * U * s) + 1e-37


def act_slope_error(z, kind):
    """The same for act_slope64: s + s c with c = z (1 - s) dt."""
    z = np.asarray(z, np.float64)
    if kind == "none":
        return np.zeros_like(z)
    if kind == "relu2":
        return 2 * U * act_slope64(z, kind)
    _, dt, s, ds = _sigmoid_parts(z, kind)
    c = np.abs(z) * (1 - s) * dt
    dc = np.abs(z) * dt * (ds + U) + 5 * U * c
    return ds * (1 + c) + s * dc + 4 * U * (s + s * c) + 1e-37
