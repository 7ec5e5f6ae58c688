"""Row-wise operators in float64: the RMS norm with the residual's addition (optionally to e4m3 with a
scale per row), the dense layer, and their gradients.  Plain NumPy; shares nothing with csrc/."""
from __future__ import annotations

import math

import numpy as np

TINY = 2.0 ** -110
DEGREE = np.array([0] + [1] * 3 + [2] * 5 + [3] * 7)      # degree of component lm


def row_weight(weight, cols: int) -> np.ndarray:
    """The weight of every column: [cols], or [4, C] per degree and channel for cols = 16 C."""
    if weight is None:
        return np.ones(cols)
    return weight if weight.ndim == 1 else weight[DEGREE].reshape(cols)


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6):
    """(y, s) of x [rows, cols]."""
    s = x if residual is None else x + residual
    return s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * row_weight(weight, s.shape[1]), s


def rms_norm_grad(g, s, weight=None, g_s=None, eps: float = 1e-6):
    """(g_x, g_weight or None)."""
    rows, cols = s.shape
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    n = s * rstd
    h = g * row_weight(weight, cols)
    g_x = rstd * (h - n * (h * n).mean(1, keepdims=True))
    if g_s is not None:
        g_x = g_x + g_s
    if weight is None:
        return g_x, None
    g_w = (g * n).sum(0)
    if weight.ndim == 2:
        parts = g_w.reshape(16, cols // 16)
        g_w = np.stack([parts[DEGREE == l].sum(0) for l in range(4)])
    return g_x, g_w


def e4m3(v):
    """v rounded to the nearest e4m3 value (ties to even, magnitudes above 448 to 448): in the binade of
    2^e, e >= -6, the values are multiples of 2^(e - 3)."""
    v = np.asarray(v, dtype=np.float64)
    e = np.clip(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -30))), -6, 8)
    step = np.exp2(e - 3)
    return np.clip(np.round(v / step) * step, -448.0, 448.0)


def scale_of(y):
    """Scale per row: max |y| / 448, or 1 where that maximum is below 2^-110."""
    top = np.abs(y).max(1)
    return np.where(top < TINY, 1.0, top / 448.0)


def activation(z, name: str):
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return z * phi(z)
    return z


def slope(z, name: str):
    if name == "silu":
        p = 1.0 / (1.0 + np.exp(-z))
        return p + z * p * (1.0 - p)
    if name == "gelu":
        return phi(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def phi(z):
    from scipy.special import erfc
    return 0.5 * erfc(-z / math.sqrt(2.0))


def dense(x, weight, bias=None, act: str = "none", residual=None):
    """(y, z) of x [rows, K], weight [N, K]."""
    z = x @ weight.T
    if bias is not None:
        z = z + bias
    y = activation(z, act)
    return (y if residual is None else y + residual), z


def dense_grad(g, x, weight, z=None, act: str = "none"):
    """(g_x, g_weight, g_bias)."""
    gz = g if z is None else g * slope(z, act)
    return gz @ weight, gz.T @ x, gz.sum(0)
