"""Refusals of the row-wise operators that the library makes on the host, before any device call."""
import ctypes

import pytest

import edge_message_passing_b200 as emp

ARG, UNSUPPORTED = -1, -8
P = 1 << 20            # a well aligned address that is never read


def norm(**kw):
    f = dict(rows=4, cols=64, dtype=0, y_dtype=0, degrees=0, eps=1e-6, x=P, ldx=64, y=P, ldy=64)
    f.update(kw)
    return emp.lib().mp_rms_norm(ctypes.byref(emp.RmsNormC(**f)), None)


def norm_grad(**kw):
    f = dict(rows=4, cols=64, dtype=0, degrees=0, eps=1e-6, g=P, ldg=64, s=P, lds=64, g_x=P, ldgx=64)
    f.update(kw)
    return emp.lib().mp_rms_norm_grad(ctypes.byref(emp.RmsNormGradC(**f)), None, 0, None)


def dense(**kw):
    f = dict(rows=4, fan_in=64, fan_out=32, dtype=0, y_dtype=0, x=P, ldx=64, weight=P, ldw=64, y=P, ldy=32)
    f.update(kw)
    return emp.lib().mp_dense(ctypes.byref(emp.DenseC(**f)), None, 0, None)


def dense_grad(**kw):
    f = dict(rows=4, fan_in=64, fan_out=32, dtype=0, g=P, ldg=32, x=P, ldx=64, weight=P, ldw=64, g_x=P, ldgx=64)
    f.update(kw)
    return emp.lib().mp_dense_grad(ctypes.byref(emp.DenseGradC(**f)), None, 0, None)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(dtype=3), dict(dtype=7), dict(y_dtype=1),
                                dict(degrees=2), dict(degrees=1, cols=40), dict(eps=0.0), dict(eps=-1.0),
                                dict(eps=float("inf")), dict(eps=float("nan")), dict(x=None), dict(y=None), dict(ldx=63),
                                dict(ldy=10), dict(x=P + 2), dict(residual=P, ldr=3), dict(s=P, lds=0), dict(weight=P + 1),
                                dict(scale=P), dict(y_dtype=3), dict(ldx=-64), dict(ldx=1 << 41)])
def test_norm(kw):
    assert norm(**kw) == ARG


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(cols=0), dict(dtype=3), dict(eps=0.0), dict(g=None), dict(s=None),
                                dict(g_x=None), dict(ldg=1), dict(g_s=P, ldgs=1), dict(weight=P + 2)])
def test_norm_gradient(kw):
    assert norm_grad(**kw) == ARG


def test_rows_too_wide():
    assert norm(cols=8193, ldx=8193, ldy=8193) == UNSUPPORTED
    assert norm_grad(cols=8193, ldg=8193, lds=8193, ldgx=8193) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(rows=(1 << 31) - 256), dict(fan_in=0), dict(fan_out=0), dict(fan_in=65537),
                                dict(fan_out=65537), dict(dtype=4), dict(dtype=0, y_dtype=1), dict(dtype=3, y_dtype=3),
                                dict(activation=3), dict(activation=-1), dict(x=None), dict(weight=None), dict(y=None),
                                dict(ldx=63), dict(ldw=63), dict(ldy=31), dict(x=P + 1), dict(bias=P + 2),
                                dict(residual=P, ldr=31), dict(z=P, ldz=31), dict(x_scale=P), dict(w_scale=P),
                                dict(dtype=3, y_dtype=1, w_scale=P), dict(dtype=3, y_dtype=1, x_scale=P)])
def test_dense(kw):
    assert dense(**kw) == ARG


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(fan_in=0), dict(fan_out=65537), dict(dtype=3), dict(activation=9),
                                dict(g=None), dict(ldg=31), dict(z=P, ldz=32), dict(activation=1), dict(weight=None),
                                dict(ldgx=63), dict(g_weight=P, x=None), dict(g_weight=P + 1), dict(g_bias=P + 3)])
def test_dense_gradient(kw):
    assert dense_grad(**kw) == ARG


def test_workspace():
    """Too small a workspace is refused before its pointer is looked at; then a null or misaligned one."""
    assert norm_grad(g_weight=P) == -6
    a = emp.DenseGradC(rows=400, fan_in=64, fan_out=32, dtype=0, g=P, ldg=32, x=P, ldx=64, weight=P, ldw=64, g_x=P, ldgx=64,
                       g_bias=P)
    L = emp.lib()
    need = L.mp_dense_grad_workspace_bytes(ctypes.byref(a))
    assert need > 0
    assert L.mp_dense_grad(ctypes.byref(a), P, need - 1, None) == -6
    assert L.mp_dense_grad(ctypes.byref(a), None, need, None) == ARG
    assert L.mp_dense_grad(ctypes.byref(a), P + 16, need, None) == ARG


def test_zero_rows_and_null():
    assert norm(rows=0, x=None, y=None) == 0 and dense(rows=0, x=None, y=None) == 0
    assert norm_grad(rows=0, g=None, s=None, g_x=None) == 0 and dense_grad(rows=0, g=None, g_x=None) == 0
    L = emp.lib()
    assert L.mp_rms_norm(None, None) == ARG and L.mp_rms_norm_grad(None, None, 0, None) == ARG
    assert L.mp_dense(None, None, 0, None) == ARG and L.mp_dense_grad(None, None, 0, None) == ARG
    assert L.mp_rms_norm_grad_workspace_bytes(None) == 0 and L.mp_dense_workspace_bytes(None) == 0
    assert L.mp_dense_grad_workspace_bytes(None) == 0
