"""Pins of the float64 row-wise operators: closed forms, invariance, finite differences."""
import math

import numpy as np
import pytest

from oracle import rows as orow
from oracle import sh


def _rng(seed):
    return np.random.default_rng(seed)


def test_norm_of_a_constant_row_and_of_zeros():
    y, s = orow.rms_norm(np.full((2, 5), 3.0), eps=1e-300)
    assert np.allclose(y, 1.0, rtol=1e-15) and np.all(s == 3.0)
    y, _ = orow.rms_norm(np.zeros((1, 4)), eps=1e-6)
    assert np.all(y == 0.0)


def test_norm_by_degree_commutes_with_rotations():
    g = _rng(1)
    C = 3
    x, w = g.standard_normal((5, 16, C)), g.standard_normal((4, C))
    D = sh.wigner_D(sh.random_rotation(g))
    norm = lambda a: orow.rms_norm(a.reshape(5, -1), w)[0].reshape(5, 16, C)  # noqa: E731
    assert np.allclose(norm(np.einsum("ab,nbc->nac", D, x)), np.einsum("ab,nbc->nac", D, norm(x)), atol=1e-12)


def test_e4m3_values():
    bits = np.arange(256)
    e, m, sign = (bits >> 3) & 15, bits & 7, np.where(bits < 128, 1.0, -1.0)
    value = sign * np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * np.exp2(e - 7.0))
    value = np.unique(value[~((e == 15) & (m == 7))])
    assert value.max() == 448.0
    assert np.array_equal(orow.e4m3(value), value)
    v = _rng(2).uniform(-500, 500, 2000) * 10.0 ** _rng(3).uniform(-6, 0, 2000)
    near = value[np.abs(v[:, None] - value[None]).argmin(1)]
    assert np.array_equal(np.abs(orow.e4m3(v) - v), np.abs(near - v))
    assert orow.e4m3(17.0) == 16.0 and orow.e4m3(19.0) == 20.0 and orow.e4m3(1e9) == 448.0      # ties to even


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_activation_slopes_by_differences(act):
    z = np.linspace(-6, 6, 101)
    d = (orow.activation(z + 1e-5, act) - orow.activation(z - 1e-5, act)) / 2e-5
    assert np.abs(d - orow.slope(z, act)).max() < 1e-9
    assert orow.activation(np.array([0.0]), act)[0] == 0.0


def test_gelu_at_one():
    assert math.isclose(orow.activation(np.array([1.0]), "gelu")[0], 0.8413447460685429, rel_tol=1e-14)


def _differences(f, a, h=1e-6):
    out = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        p, m = a.copy(), a.copy()
        p[i] += h
        m[i] -= h
        out[i] = (f(p) - f(m)) / (2 * h)
    return out


@pytest.mark.parametrize("degrees", [False, True])
def test_norm_gradient_by_differences(degrees):
    g = _rng(4)
    rows, cols = 3, 32
    s, w = g.standard_normal((rows, cols)), g.standard_normal((4, 2) if degrees else (cols,))
    gy, gs = g.standard_normal((rows, cols)), g.standard_normal((rows, cols))
    loss = lambda s_, w_: (orow.rms_norm(s_, w_, eps=0.1)[0] * gy).sum() + (s_ * gs).sum()  # noqa: E731
    g_x, g_w = orow.rms_norm_grad(gy, s, w, gs, eps=0.1)
    assert np.abs(g_x - _differences(lambda a: loss(a, w), s)).max() < 1e-8
    assert np.abs(g_w - _differences(lambda a: loss(s, a), w)).max() < 1e-8


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_dense_gradient_by_differences(act):
    g = _rng(5)
    x, w, b, gy = (g.standard_normal(s) for s in ((4, 5), (3, 5), (3,), (4, 3)))
    loss = lambda x_, w_, b_: (orow.dense(x_, w_, b_, act)[0] * gy).sum()  # noqa: E731
    z = orow.dense(x, w, b, act)[1]
    g_x, g_w, g_b = orow.dense_grad(gy, x, w, None if act == "none" else z, act)
    assert np.abs(g_x - _differences(lambda a: loss(a, w, b), x)).max() < 1e-8
    assert np.abs(g_w - _differences(lambda a: loss(x, a, b), w)).max() < 1e-8
    assert np.abs(g_b - _differences(lambda a: loss(x, w, a), b)).max() < 1e-8
