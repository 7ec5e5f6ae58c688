"""The row-wise operators over the rest of their range, against the float64 oracle: forms that take several tiles per
block, values at the ends of the types, long sums.  Tolerances as derived in test_gpu_rows.py where nothing else is said."""
import numpy as np
import pytest

from test_gpu_rows import TYPES, dense_tol, dev, host, near, normal, to_e4m3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import edge_message_passing_b200 as emp  # noqa: E402


# ------------------------------------------------------------------ several tiles per block
ROWS = 2 * 148 * 128 + 2200 + 77            # more than two tiles of 128 rows for every SM, the last one ragged


@pytest.mark.parametrize("K,N", [(100, 132), (200, 64), (515, 40), (128, 61)])
@pytest.mark.parametrize("act,residual,keep", [("none", False, False), ("silu", True, False), ("gelu", True, True),
                                               ("silu", False, True)])
def test_fp32_of_a_long_k_and_many_tiles(K, N, act, residual, keep):
    """k above 96, whose sums are held in registers: whole rows by TMA (N = 132, 64, 40) and by columns (61)."""
    rng = np.random.default_rng(K + N)
    t = torch.float32
    x, w, b = dev(normal(rng, ROWS, K), t), dev(normal(rng, N, K) / np.sqrt(K), t), dev(normal(rng, N), t)
    r = dev(normal(rng, ROWS, N), t) if residual else None
    out = emp.mp_dense(x, w, b, activation=act, residual=r, keep_z=keep)
    y, z = out if keep else (out, None)
    ry, rz, ty, tz = dense_tol(host(x), host(w), host(b), host(r), act, t, K)
    near(y, ry, ty, "y")
    if keep:
        near(z, rz, tz, "z")
    assert emp.last_device_error() == 0


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("K,N", [(144, 96), (400, 264), (100, 61)])
@pytest.mark.parametrize("act,residual,keep", [("none", False, False), ("gelu", True, False), ("gelu", True, True),
                                               ("silu", False, True)])
def test_8_bits_of_many_tiles(K, N, act, residual, keep, out):
    t, rng = TYPES[out], np.random.default_rng(K + N)
    (x, xs), (w, ws) = to_e4m3(normal(rng, ROWS, K) * np.exp(normal(rng, ROWS, 1))), to_e4m3(normal(rng, N, K) / np.sqrt(K))
    b = dev(normal(rng, N), torch.float32)
    r = dev(normal(rng, ROWS, N), t) if residual else None
    res = emp.mp_dense(x, w, b, activation=act, residual=r, x_scale=xs, w_scale=ws, out_dtype=t, keep_z=keep)
    y, z = res if keep else (res, None)
    ry, rz, ty, tz = dense_tol(host(x) * host(xs)[:, None], host(w) * host(ws)[:, None], host(b), host(r), act, t, K)
    near(y, ry, ty, "y")
    if keep:
        near(z, rz, tz, "z")
    assert emp.last_device_error() == 0


@pytest.mark.parametrize("rows,K,N", [(3, 17, 5), (16, 48, 96), (129, 128, 250), (300, 2048, 72)])
def test_gelu_of_8_bits(rows, K, N):
    rng = np.random.default_rng(rows + K + N)
    (x, xs), (w, ws) = to_e4m3(normal(rng, rows, K)), to_e4m3(normal(rng, N, K) / np.sqrt(K))
    for t in TYPES.values():
        y, z = emp.mp_dense(x, w, activation="gelu", x_scale=xs, w_scale=ws, out_dtype=t, keep_z=True)
        ry, rz, ty, tz = dense_tol(host(x) * host(xs)[:, None], host(w) * host(ws)[:, None], None, None, "gelu", t, K)
        near(z, rz, tz, "z")
        near(y, ry, ty, "y")
