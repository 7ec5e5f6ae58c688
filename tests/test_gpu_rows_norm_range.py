"""Norms of rows of large values (|s| up to 1e18, whose sum of squares passes FP32's range from 341 columns on), against the
float64 oracle, in every form of the kernels: rows of 16-byte vectors, contiguous rows off 16 bytes, pitched rows off 16
bytes; with ordinary, infinite and NaN rows between them.  Tolerances as derived in test_gpu_rows.py."""
import numpy as np
import pytest

from oracle import rows as orow
from test_gpu_rows import EPS, TYPES, U, dev, half_step, host, near, normal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import edge_message_passing_b200 as emp  # noqa: E402

# (rows, columns, pitch - columns, per degree)
FORMS = [(7, 64, 0, False), (6, 512, 0, False), (700, 1024, 0, False), (5, 2048, 0, True), (4, 8192, 0, False),     # vectors
         (9, 515, 0, False), (40, 1001, 0, False), (3, 2047, 0, False), (3000, 66, 0, False), (5, 16 * 35, 0, True),  # contiguous
         (9, 515, 3, False), (40, 1001, 5, False), (3, 8191, 0, False), (4, 8190, 3, False), (700, 66, 3, False),     # any
         (6, 90, 1, False)]


def view(a, pad, t):
    rows, cols = a.shape
    full = torch.zeros(rows * (cols + pad), dtype=t, device="cuda")
    v = torch.as_strided(full, (rows, cols), (cols + pad, 1))
    v.copy_(dev(a, t))
    return v


def big_rows(rng, rows, cols, top):
    """Rows of magnitudes up to `top`, every third one an ordinary row; one row is `top` throughout."""
    a = rng.uniform(-1, 1, (rows, cols)) * np.where(np.arange(rows) % 3 == 1, 1.0, top)[:, None]
    a[0] = top
    return a


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("top", [1e15, 1e18])
@pytest.mark.parametrize("rows,cols,pad,degrees", FORMS)
def test_norm_of_large_values(rows, cols, pad, degrees, top, type):
    t, rng = TYPES[type], np.random.default_rng(rows + cols)
    w = dev(1 + 0.3 * normal(rng, *((4, cols // 16) if degrees else (cols,))), t)
    for x, r in ((view(big_rows(rng, rows, cols, top), pad, t), None),
                 (view(big_rows(rng, rows, cols, 0.6 * top), pad, t), view(big_rows(rng, rows, cols, 0.4 * top), pad, t))):
        for weight in (w, None):
            ry, rs = orow.rms_norm(host(x), host(weight), host(r), EPS)
            y, s = emp.mp_rms_norm(x, weight, residual=r, eps=EPS)
            near(y, ry, (half_step(t) + 32 * U) * np.abs(ry) + 1e-37, "y")
            near(s, rs, (half_step(t) + U) * np.abs(rs), "s")
            q, scale, _ = emp.mp_rms_norm(x, weight, residual=r, eps=EPS, quantize=True)
            rscale = orow.scale_of(ry)
            near(scale, rscale, 40 * U * rscale, "scale")
            value = host(q) * host(scale)[:, None]
            assert np.all(np.abs(value - ry) <= np.maximum(2.0 ** -4 * np.abs(ry), 2.0 ** -10 * rscale[:, None])
                          + 64 * U * np.abs(ry))


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("top", [1e15, 1e18])
@pytest.mark.parametrize("rows,cols,pad,degrees", FORMS)
def test_norm_gradient_of_large_values(rows, cols, pad, degrees, top, type):
    t, rng = TYPES[type], np.random.default_rng(rows + cols + 1)
    s, g = view(big_rows(rng, rows, cols, top), pad, t), view(normal(rng, rows, cols), pad, t)
    gs = view(normal(rng, rows, cols), pad, t)
    w = dev(1 + 0.3 * normal(rng, *((4, cols // 16) if degrees else (cols,))), t)
    S, G, W = host(s), host(g), host(w)
    rstd = 1 / np.sqrt((S * S).mean(1, keepdims=True) + EPS)
    n, h = S * rstd, G * orow.row_weight(W, cols)
    for through in (None, gs):
        g_x, g_w = emp.mp_rms_norm_grad(g, s, w, g_s=through, eps=EPS)
        rx, rw = orow.rms_norm_grad(G, S, W, host(through), EPS)
        size = rstd * (np.abs(h) + np.abs(n) * np.abs(h * n).mean(1, keepdims=True)) + (0 if through is None else np.abs(host(gs)))
        near(g_x, rx, half_step(t) * np.abs(rx) + 64 * U * size, "g_x")
        total = np.abs(G * n).sum(0)
        if degrees:
            total = np.stack([total.reshape(16, -1)[orow.DEGREE == l].sum(0) for l in range(4)])
        near(g_w, rw, half_step(t) * np.abs(rw) + (rows / 592 + 400) * U * total, "g_w")


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows,cols,pad,degrees", FORMS)
def test_infinite_and_nan_rows_stay_alone(rows, cols, pad, degrees, type):
    """An infinite element: itself NaN, the row's others zero; a NaN: the whole row; in 8 bits both rows NaN.  The other rows
    have the bits that they have without them."""
    t, rng = TYPES[type], np.random.default_rng(rows * cols)
    a = normal(rng, rows, cols)
    clean = view(a, pad, t)
    bad = clean.clone() if pad == 0 else view(a, pad, t)
    bad[0, cols // 2] = float("inf")
    bad[2, 1] = float("nan")
    y0, y = emp.mp_rms_norm(clean, eps=EPS)[0], emp.mp_rms_norm(bad, eps=EPS)[0]
    rest = [i for i in range(rows) if i not in (0, 2)]
    assert torch.equal(y[rest], y0[rest]) and torch.isnan(y[2]).all()
    assert torch.isnan(y[0, cols // 2]) and torch.count_nonzero(y[0]) == 1
    q, scale, _ = emp.mp_rms_norm(bad, eps=EPS, quantize=True)
    q0, scale0, _ = emp.mp_rms_norm(clean, eps=EPS, quantize=True)
    assert torch.isnan(q[[0, 2]].float()).all() and torch.isnan(scale[[0, 2]]).all()
    assert torch.equal(q[rest].view(torch.uint8), q0[rest].view(torch.uint8)) and torch.equal(scale[rest], scale0[rest])
    g = view(normal(rng, rows, cols), pad, t)
    g0, gx = emp.mp_rms_norm_grad(g, clean, eps=EPS)[0], emp.mp_rms_norm_grad(g, bad, eps=EPS)[0]
    assert torch.equal(gx[rest], g0[rest]) and torch.isnan(gx[2]).all() and not torch.isfinite(gx[0]).all()
