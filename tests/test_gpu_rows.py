"""The row-wise operators on the GPU against the float64 oracle (oracle/rows.py).

Tolerances, element by element, with u = 2^-24 (half a step of FP32) and e = finfo(type).eps / 2 (half a
step of the output's type; fp16 below its normal range: an absolute 2^-25):

* norm: s is one FP32 addition; the sum of squares has at most 16 + 5 + 16 additions in a row of a
  thread, a warp and the warps, halved by the root, and rsqrt, the mean and two products a few u:
  |dy| <= (e + 32 u) |y|.
* norm's gradient: the same 37 additions in each of the two means:
  |dg_x| <= e |g_x| + 64 u (|g_s| + rstd (|h| + |n| mean|h n|)).
  g_w sums rows one after the other (at most rows / 592 + 1 of them per thread), then row groups, warps
  and blocks (at most 8 + 37 + 16, times 7 components): |dg_w| <= e |g_w| + (rows / 592 + 400) u sum|g n|.
* dense: 16- and 8-bit products are exact in FP32; an FP32 product in 3xTF32 drops less than 3 * 2^-22 of
  it.  Each of the K products is added with an error of at most 2 u of the running sum (a truncating
  adder): |dz| <= e |z| + (2^-20 + 2 (K + 8) u) S + 4 u |b|, S = sum|x w|, and, the slope of either
  activation being below 1.13, |dy| <= e |y| + 1.13 |dz| + 16 u (|z| + |y|).
* dense's gradient: gz is rounded to the operands' type (e) in both products:
  |d| <= e |ref| + (e + 2^-20 + 2 (n + 8) u) sum|terms| over the n summed terms, where without an
  activation gz is g and unrounded.
"""
import ctypes

import numpy as np
import pytest

import synth
from oracle import rows as orow

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import edge_message_passing_b200 as emp  # noqa: E402

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def half_step(t):
    return torch.finfo(t).eps / 2


def floor_of(t):
    return 2.0 ** -25 if t == torch.float16 else 1e-37


def dev(a, t):
    return torch.from_numpy(np.asarray(a)).cuda().to(t)


def host(t):
    return None if t is None else t.double().cpu().numpy()


def near(got, ref, tol, what=""):
    d = np.abs(host(got).reshape(ref.shape) - ref)
    assert np.all(d <= tol), f"{what}: {(d - tol).max()} over, {np.argwhere(d > tol)[:3].tolist()}"


def normal(rng, *shape):
    return rng.standard_normal(shape)


# ------------------------------------------------------------------ norm
NORM_SHAPES = [(1, 1), (3, 2), (5, 7), (64, 31), (2, 33), (17, 128), (1, 515), (9, 1000), (700, 96), (3, 4097), (2, 8191),
               (5, 8192)]


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_per_column(rows, cols, type, residual):
    t, rng = TYPES[type], np.random.default_rng(rows * 10007 + cols)
    x = dev(normal(rng, rows, cols) * np.exp(normal(rng, rows, 1)), t)
    r = dev(normal(rng, rows, cols), t) if residual else None
    w = dev(1 + 0.3 * normal(rng, cols), t) if cols % 2 else None
    y, s = emp.mp_rms_norm(x, w, residual=r, eps=EPS)
    ry, rs = orow.rms_norm(host(x), host(w), host(r), EPS)
    near(y, ry, (half_step(t) + 32 * U) * np.abs(ry) + floor_of(t), "y")
    near(s, rs, (half_step(t) + U) * np.abs(rs) + floor_of(t), "s")
    if r is None:
        assert s is x


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows,C", [(1, 1), (3, 5), (64, 64), (33, 128), (2, 256), (700, 32), (5, 512)])
def test_norm_per_degree(rows, C, type):
    t, rng = TYPES[type], np.random.default_rng(rows * 101 + C)
    x, r, w = dev(normal(rng, rows, 16, C), t), dev(normal(rng, rows, 16, C), t), dev(1 + 0.3 * normal(rng, 4, C), t)
    y, s = emp.mp_rms_norm(x, w, residual=r, eps=EPS)
    ry, rs = orow.rms_norm(host(x).reshape(rows, -1), host(w), host(r).reshape(rows, -1), EPS)
    assert y.shape == s.shape == x.shape
    near(y, ry, (half_step(t) + 32 * U) * np.abs(ry) + floor_of(t), "y")
    near(s, rs, (half_step(t) + U) * np.abs(rs) + floor_of(t), "s")
    flat, _ = emp.mp_rms_norm(x.view(rows, 16 * C), w, residual=r.view(rows, 16 * C), eps=EPS)
    assert torch.equal(flat.view_as(y), y)


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows,cols,degrees", [(1, 1, False), (5, 33, False), (3, 1000, False), (200, 16 * 32, True),
                                               (7, 16 * 128, True), (2, 8192, False), (4, 16 * 3, True)])
def test_norm_to_8_bits(rows, cols, degrees, type):
    """q scale is within half an e4m3 step of y (2^-4 of the value, 2^-10 of the scale below the normal
    range), and y itself within the norm's tolerance; the largest element is stored as +-448."""
    t, rng = TYPES[type], np.random.default_rng(cols)
    x, r = dev(normal(rng, rows, cols), t), dev(normal(rng, rows, cols), t)
    w = dev(1 + 0.3 * normal(rng, *((4, cols // 16) if degrees else (cols,))), t)
    q, scale, s = emp.mp_rms_norm(x, w, residual=r, eps=EPS, quantize=True)
    assert q.dtype == torch.float8_e4m3fn and scale.shape == (rows,) and scale.dtype == torch.float32
    ry, rs = orow.rms_norm(host(x), host(w), host(r), EPS)
    rscale = orow.scale_of(ry)
    near(scale, rscale, 40 * U * rscale, "scale")
    near(s, rs, (half_step(t) + U) * np.abs(rs) + floor_of(t), "s")
    value = host(q) * host(scale)[:, None]
    assert np.all(np.abs(value - ry) <= np.maximum(2.0 ** -4 * np.abs(ry), 2.0 ** -10 * rscale[:, None]) + 64 * U * np.abs(ry))
    # away from the borders of the rounding it is the oracle's value
    u = ry / rscale[:, None]
    border = np.abs(orow.e4m3(u * (1 + 64 * U)) - orow.e4m3(u * (1 - 64 * U))) > 0
    assert np.array_equal(host(q)[~border], orow.e4m3(u)[~border])
    assert np.all(np.abs(host(q)).max(1) == 448.0)


def test_norm_rows_of_zeros_tiny_values_nan_and_infinity():
    x = torch.zeros((6, 64), device="cuda")
    x[1] = 1e-30
    x[2, 3] = float("nan")
    x[3, 5] = float("inf")
    x[4] = 2.0
    x[5] = 1e18
    y, _ = emp.mp_rms_norm(x, eps=EPS)
    assert torch.all(y[0] == 0) and torch.allclose(y[1], torch.full_like(y[1], 1e-27), rtol=1e-5)
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, 5]) and torch.all(y[3, 6:] == 0)
    assert torch.allclose(y[4:], torch.ones_like(y[4:]), rtol=1e-5)
    q, scale, _ = emp.mp_rms_norm(x, eps=EPS, quantize=True)
    assert torch.all(q[0].float() == 0) and scale[0] == 1
    assert torch.isnan(q[2].float()).all() and torch.isnan(scale[2]) and torch.isnan(q[3].float()).all()
    assert torch.all(q[4].float() == 448)
    tiny = torch.full((1, 64), 1e-33, device="cuda")
    q, scale, _ = emp.mp_rms_norm(tiny, torch.full((64,), 1e-5, device="cuda"), eps=EPS, quantize=True)
    assert scale[0] == 1 and torch.all(q.float() == 0)


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows,cols,degrees,through", [(1, 1, False, False), (3, 7, False, True), (5, 33, False, True),
                                                       (1300, 96, False, True), (2, 8192, False, False), (9, 4097, False, True),
                                                       (64, 16 * 64, True, True), (700, 16 * 32, True, False),
                                                       (3, 16 * 3, True, True), (2500, 16 * 8, True, True)])
def test_norm_gradient(rows, cols, degrees, through, type):
    t, rng = TYPES[type], np.random.default_rng(rows + cols)
    s, g = dev(normal(rng, rows, cols) * np.exp(normal(rng, rows, 1)), t), dev(normal(rng, rows, cols), t)
    gs = dev(normal(rng, rows, cols), t) if through else None
    w = dev(1 + 0.3 * normal(rng, *((4, cols // 16) if degrees else (cols,))), t)
    g_x, g_w = emp.mp_rms_norm_grad(g, s, w, g_s=gs, eps=EPS)
    S, G, W = host(s), host(g), host(w)
    rx, rw = orow.rms_norm_grad(G, S, W, host(gs), EPS)
    rstd = 1 / np.sqrt((S * S).mean(1, keepdims=True) + EPS)
    n, h = S * rstd, G * orow.row_weight(W, cols)
    size = rstd * (np.abs(h) + np.abs(n) * np.abs(h * n).mean(1, keepdims=True)) + (0 if gs is None else np.abs(host(gs)))
    near(g_x, rx, half_step(t) * np.abs(rx) + 64 * U * size + floor_of(t), "g_x")
    total = np.abs(G * n).sum(0)
    if degrees:
        total = np.stack([total.reshape(16, -1)[orow.DEGREE == l].sum(0) for l in range(4)])
    near(g_w, rw, half_step(t) * np.abs(rw) + (rows / 592 + 400) * U * total + floor_of(t), "g_w")
    g_x2, g_w2 = emp.mp_rms_norm_grad(g, s, w, g_s=gs, eps=EPS)
    assert torch.equal(g_x, g_x2) and torch.equal(g_w, g_w2)
    only_x, none = emp.mp_rms_norm_grad(g, s, None, g_s=gs, eps=EPS)
    assert none is None
    ox = orow.rms_norm_grad(G, S, None, host(gs), EPS)[0]
    size1 = rstd * (np.abs(G) + np.abs(n) * np.abs(G * n).mean(1, keepdims=True)) + (0 if gs is None else np.abs(host(gs)))
    near(only_x, ox, half_step(t) * np.abs(ox) + 64 * U * size1 + floor_of(t), "g_x without a weight")


def test_norm_gradient_by_differences():
    """dE/dx of E = sum(y gy) + sum(s gs) by central differences of the forward in FP32: the step 2^-7
    leaves h^2 / 6 |E'''| and rounding of E / h, both below 2e-3 of the largest gradient here."""
    rng = np.random.default_rng(3)
    x, gy = dev(normal(rng, 1, 32), torch.float32), dev(normal(rng, 1, 32), torch.float32)
    w = dev(1 + 0.3 * normal(rng, 32), torch.float32)
    h = 2.0 ** -7
    steps = torch.cat([x + h * torch.eye(32, device="cuda"), x - h * torch.eye(32, device="cuda")])
    y, _ = emp.mp_rms_norm(steps, w, eps=0.1)
    E = (y.double() * gy.double()).sum(1)
    d = (E[:32] - E[32:]) / (2 * h)
    g_x, _ = emp.mp_rms_norm_grad(gy, x, w, eps=0.1)
    assert (g_x.double()[0] - d).abs().max() <= 2e-3 * d.abs().max()


# ------------------------------------------------------------------ dense
def dense_tol(x, w, b, r, act, t, K, extra=0.0):
    y, z = orow.dense(x, w, b, act, r)
    S = np.abs(x) @ np.abs(w).T
    dz = (2.0 ** -20 + 2 * (K + 8) * U) * S + 4 * U * (0 if b is None else np.abs(b))
    tz = half_step(t) * np.abs(z) + dz + floor_of(t)
    ty = half_step(t) * np.abs(y) + 1.13 * dz + 16 * U * (np.abs(z) + np.abs(y)) + floor_of(t)
    return y, z, ty, tz


DENSE_SHAPES = [(1, 1, 1), (1, 64, 128), (1, 2500, 40), (16, 2000, 1500), (5, 70, 9000), (3, 7, 5), (8, 256, 1024), (9, 100, 33), (17, 515, 250), (64, 64, 64),
                (127, 32, 8), (128, 128, 128), (129, 130, 131), (257, 96, 512), (1000, 48, 25), (300, 2048, 72),
                (2, 1100, 1000), (640, 64, 700)]


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows,K,N", DENSE_SHAPES)
@pytest.mark.parametrize("act,bias,residual", [("none", False, False), ("silu", True, True), ("gelu", True, False)])
def test_dense(rows, K, N, type, act, bias, residual):
    t, rng = TYPES[type], np.random.default_rng(rows * 31 + K * 7 + N)
    x, w = dev(normal(rng, rows, K), t), dev(normal(rng, N, K) / np.sqrt(K), t)
    b = dev(normal(rng, N), t) if bias else None
    r = dev(normal(rng, rows, N), t) if residual else None
    y, z = emp.mp_dense(x, w, b, activation=act, residual=r, keep_z=True)
    ry, rz, ty, tz = dense_tol(host(x), host(w), host(b), host(r), act, t, K)
    near(z, rz, tz, "z")
    near(y, ry, ty, "y")
    assert torch.equal(emp.mp_dense(x, w, b, activation=act, residual=r), y)


def to_e4m3(a):
    scale = torch.from_numpy(orow.scale_of(a)).float().cuda()
    return (torch.from_numpy(a).cuda() / scale.double()[:, None]).to(torch.float8_e4m3fn), scale


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("rows,K,N", [(1, 1, 1), (3, 17, 5), (8, 256, 128), (16, 48, 96), (129, 128, 250), (300, 2048, 72),
                                      (1000, 100, 130)])
@pytest.mark.parametrize("act,bias,residual", [("none", False, False), ("silu", True, True)])
def test_dense_of_8_bits(rows, K, N, out, act, bias, residual):
    t, rng = TYPES[out], np.random.default_rng(rows + K + N)
    x, xs = to_e4m3(normal(rng, rows, K) * np.exp(normal(rng, rows, 1)))
    w, ws = to_e4m3(normal(rng, N, K) / np.sqrt(K))
    b = dev(normal(rng, N), torch.float32) if bias else None
    r = dev(normal(rng, rows, N), t) if residual else None
    y, z = emp.mp_dense(x, w, b, activation=act, residual=r, x_scale=xs, w_scale=ws, out_dtype=t, keep_z=True)
    X, W = host(x) * host(xs)[:, None], host(w) * host(ws)[:, None]
    ry, rz, ty, tz = dense_tol(X, W, host(b), host(r), act, t, K)
    near(z, rz, tz, "z")
    near(y, ry, ty, "y")


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows,K,N", [(1, 1, 1), (1, 64, 128), (3, 7, 5), (17, 515, 250), (128, 128, 128), (129, 130, 131),
                                      (1000, 48, 25), (2500, 64, 72), (640, 200, 512), (5000, 33, 9), (300, 512, 1024)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_dense_gradient(rows, K, N, type, act):
    t, rng = TYPES[type], np.random.default_rng(rows * 3 + K + N)
    x, w, g = dev(normal(rng, rows, K), t), dev(normal(rng, N, K) / np.sqrt(K), t), dev(normal(rng, rows, N), t)
    z = None if act == "none" else dev(2 * normal(rng, rows, N), t)
    X, W, G, Z = host(x), host(w), host(g), host(z)
    g_x, g_w, g_b = emp.mp_dense_grad(g, x, w, z=z, activation=act)
    rx, rw, rb = orow.dense_grad(G, X, W, Z, act)
    gz = np.abs(G if Z is None else G * orow.slope(Z, act))
    # FP32 slopes: a few u of g times at most 1.13 and of the two terms of the slope, |z| below 12
    slack = gz + (0 if Z is None else 16 * U * np.abs(G) * (1 + np.abs(Z)))
    e = 0.0 if Z is None else half_step(t)
    f = floor_of(t)

    def tol(ref, S, n):
        return half_step(t) * np.abs(ref) + (e + 2.0 ** -20 + 2 * (n + 8) * U) * S + f * (1 + n)

    near(g_x, rx, tol(rx, slack @ np.abs(W), N) + (slack - gz) @ np.abs(W), "g_x")
    near(g_w, rw, tol(rw, slack.T @ np.abs(X), rows) + (slack - gz).T @ np.abs(X), "g_w")
    near(g_b, rb, tol(rb, slack.sum(0), rows) + (slack - gz).sum(0), "g_b")
    again = emp.mp_dense_grad(g, x, w, z=z, activation=act)
    assert all(torch.equal(a, b) for a, b in zip((g_x, g_w, g_b), again))
    for need in ("x", "weight", "bias"):
        part = emp.mp_dense_grad(g, x, w, z=z, activation=act, need_x=need == "x", need_weight=need == "weight",
                                 need_bias=need == "bias")
        for got, all_, name in zip(part, (g_x, g_w, g_b), ("x", "weight", "bias")):
            assert torch.equal(got, all_) if name == need else got is None


def test_dense_gradient_by_differences():
    """dE/dx and dE/dW of E = sum(y gy) by central differences of the forward in FP32 (step 2^-6): the cubic
    term and the rounding of E / h are below 5e-3 of the largest gradient here."""
    rng = np.random.default_rng(8)
    K, N, h = 16, 24, 2.0 ** -6
    x, w, b, gy = (dev(normal(rng, *s), torch.float32) for s in ((1, K), (N, K), (N,), (1, N)))
    w = w / 4
    _, z = emp.mp_dense(x, w, b, activation="silu", keep_z=True)
    g_x, g_w, g_b = emp.mp_dense_grad(gy, x, w, z=z, activation="silu")
    step = h * torch.eye(K, device="cuda")
    E = (emp.mp_dense(torch.cat([x + step, x - step]), w, b, activation="silu").double() * gy.double()).sum(1)
    d = (E[:K] - E[K:]) / (2 * h)
    assert (g_x.double()[0] - d).abs().max() <= 5e-3 * d.abs().max()
    d = torch.empty(N, dtype=torch.float64, device="cuda")
    for n in range(N):
        e = torch.zeros(N, device="cuda")
        e[n] = h
        p, m = (emp.mp_dense(x, w, bb, activation="silu").double() for bb in (b + e, b - e))
        d[n] = ((p - m) * gy.double()).sum() / (2 * h)
    assert (g_b.double() - d).abs().max() <= 5e-3 * d.abs().max()
    assert torch.allclose(g_w, g_b[:, None] * x, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("type", list(TYPES))
def test_non_finite_inputs_stay_in_their_row_and_column(type):
    t, rng = TYPES[type], np.random.default_rng(9)
    x, w = dev(normal(rng, 200, 64), t), dev(normal(rng, 136, 64), t)
    clean = emp.mp_dense(x, w)
    xb, wb = x.clone(), w.clone()
    xb[7, 3], xb[150, 60], wb[9, 5], wb[100, 2] = float("nan"), float("inf"), float("inf"), float("nan")
    bad = emp.mp_dense(xb, wb)
    assert not torch.isfinite(bad[[7, 150]]).any() and not torch.isfinite(bad[:, [9, 100]]).any()
    keep = torch.ones_like(clean, dtype=torch.bool)
    keep[[7, 150]] = False
    keep[:, [9, 100]] = False
    assert torch.equal(bad[keep], clean[keep])


# ------------------------------------------------------------------ layouts, streams, graphs
def _ops(x, w, wn, r):
    """One call of each operator, all outputs."""
    y, s = emp.mp_rms_norm(x, wn, residual=r)
    q, scale, _ = emp.mp_rms_norm(x, wn, residual=r, quantize=True)
    h, z = emp.mp_dense(x, w, activation="silu", keep_z=True)
    g_x, g_w = emp.mp_rms_norm_grad(y, s, wn, g_s=x)
    return (y, s, q.float(), scale, h, z, g_x, g_w, *emp.mp_dense_grad(h, x, w, z=z, activation="silu"))


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("layout", ["pitched", "offset", "transposed", "expanded"])
def test_layouts_give_the_contiguous_result(layout, type):
    t, rng = TYPES[type], np.random.default_rng(11)
    rows, K, N = 150, 72, 40
    base = dev(normal(rng, rows, 16, K), t)
    w, wn, r = dev(normal(rng, N, K), t), dev(normal(rng, K), t), dev(normal(rng, rows, K), t)
    if layout == "pitched":                    # the degree-0 channels of node features
        x = base[:, 0, :]
    elif layout == "offset":                   # one element past a 16-byte boundary
        x = base.flatten()[1:1 + rows * K].view(rows, K)
        w = torch.cat([w.flatten()[:1], w.flatten()])[1:].view(N, K)
        wn = torch.cat([wn[:1], wn])[1:]
    elif layout == "transposed":
        x = base[:K, 0, :].reshape(K, K).t()
        rows, r = K, r[:K]
    else:
        x = base[:1, 0, :].expand(rows, K)
    got = _ops(x, w, wn, r)
    ref = _ops(x.contiguous().clone(), w.clone(), wn.clone(), r)
    for i, (a, b) in enumerate(zip(got, ref)):
        # other alignment, other vector width: the sums' order may differ, so rounding may
        scale = max(1e-6, b.double().abs().max().item())
        assert (a.double() - b.double()).abs().max().item() <= (4 * half_step(t) + 1e-5 + (0.07 if i == 2 else 0)) * scale, i


def test_leading_dimensions_and_zero_rows():
    x, w = torch.randn((3, 5, 64), device="cuda"), torch.randn((32, 64), device="cuda")
    y, z = emp.mp_dense(x, w, activation="gelu", keep_z=True)
    assert y.shape == (3, 5, 32)
    assert torch.equal(y.view(15, 32), emp.mp_dense(x.view(15, 64), w, activation="gelu"))
    g_x, g_w, g_b = emp.mp_dense_grad(y, x, w, z=z, activation="gelu")
    assert g_x.shape == x.shape and g_w.shape == w.shape and g_b.shape == (32,)
    e = x[:0]
    y, z = emp.mp_dense(e, w, activation="gelu", keep_z=True)
    assert y.shape == (0, 5, 32)
    g_x, g_w, g_b = emp.mp_dense_grad(y, e, w, z=z, activation="gelu")
    assert g_x.shape == e.shape and torch.all(g_w == 0) and torch.all(g_b == 0)
    wn = torch.ones(64, device="cuda")
    q, scale, s = emp.mp_rms_norm(e, wn, residual=e, quantize=True)
    assert q.shape == e.shape and scale.shape == (0, 5) and s.shape == e.shape
    g_x, g_w = emp.mp_rms_norm_grad(e, e, wn)
    assert g_x.shape == e.shape and torch.all(g_w == 0)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_nothing_beside_the_outputs_is_written(t):
    """Through the C ABI with pitched outputs inside a larger buffer full of sentinels."""
    rng = np.random.default_rng(13)
    rows, K, N, pad = 131, 70, 45, 3
    x, w = dev(normal(rng, rows, K), t), dev(normal(rng, N, K), t)
    code = {torch.float32: 0, torch.bfloat16: 1}[t]
    st = torch.cuda.current_stream().cuda_stream
    L = emp.lib()

    def framed(c):
        full = torch.full((rows + 4, c + pad), -77.0, dtype=t, device="cuda")
        return full, full[2:2 + rows, 1:1 + c]

    def untouched(full, inner, ref):
        assert torch.equal(inner, ref)
        inner.fill_(-77.0)
        assert torch.all(full == -77.0)

    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    yf, y = framed(N)
    zf, z = framed(N)
    a = emp.DenseC(rows, K, N, code, code, 1, x.data_ptr(), K, None, w.data_ptr(), K, None, None, None, 0, y.data_ptr(),
                   N + pad, z.data_ptr(), N + pad)
    assert L.mp_dense(ctypes.byref(a), ws.data_ptr(), ws.numel(), st) == 0
    ry, rz = emp.mp_dense(x, w, activation="silu", keep_z=True)
    untouched(yf, y, ry)
    untouched(zf, z, rz)
    gf, gx = framed(K)
    d = emp.DenseGradC(rows, K, N, code, 0, ry.data_ptr(), N, None, 0, x.data_ptr(), K, w.data_ptr(), K, gx.data_ptr(),
                       K + pad, None, None)
    assert L.mp_dense_grad(ctypes.byref(d), ws.data_ptr(), ws.numel(), st) == 0
    untouched(gf, gx, emp.mp_dense_grad(ry, x, w)[0])
    yf, y = framed(K)
    sf, s = framed(K)
    n = emp.RmsNormC(rows, K, code, code, 0, 1e-6, x.data_ptr(), K, x.data_ptr(), K, None, y.data_ptr(), K + pad, None,
                     s.data_ptr(), K + pad)
    assert L.mp_rms_norm(ctypes.byref(n), st) == 0
    ry, rs = emp.mp_rms_norm(x, residual=x)
    untouched(sf, s, rs)
    assert (y.double() - ry.double()).abs().max() <= 4 * half_step(t) * ry.double().abs().max()
    y.fill_(-77.0)
    assert torch.all(yf == -77.0)


def test_two_streams_at_once_and_two_graphs():
    """The same calls on two streams, and captured in two graphs replayed in turn, give the eager bits."""
    rng = np.random.default_rng(17)
    sets = [(dev(normal(rng, 700, 128), torch.float32), dev(normal(rng, 96, 128), torch.float32),
             dev(normal(rng, 128), torch.float32), dev(normal(rng, 700, 128), torch.float32)) for _ in range(2)]
    eager = [_ops(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = _ops(*sets[i])
    torch.cuda.synchronize()
    for a, b in zip(eager, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_ops(*s))
        graphs.append(g)
    for o in outs:
        for p in o:
            p.fill_(0)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, outs):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    sets[0][0].copy_(sets[1][0])              # a replay reads the inputs anew
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs[0], _ops(*sets[0])))
    assert emp.last_device_error() == 0


# ------------------------------------------------------------------ together, between two layers
@pytest.mark.parametrize("quantize", [False, True])
def test_a_node_block_between_two_layers(quantize):
    """mp_forward, then x + agg normed per degree, a two-layer feed-forward on the degree-0 channels with its
    own residual, and mp_forward again, against the same block from the oracle's operators on the GPU
    layers' outputs; without 8 bits also the block's gradients."""
    w = synth.small_workload(ncell=1, C=32, n_layers=2, gated=True, sigma=0.1, cohort_edges=256)
    st, C = w.structure, 32
    g = emp.nl_build(torch.from_numpy(st.pos).cuda(), st.box, w.spec.cutoff)
    model, sp = emp.Model(w.spec, w.weights), torch.from_numpy(st.species).cuda()
    rng = np.random.default_rng(19)
    x = dev(normal(rng, g.n_atoms, 16, C), torch.float32)
    wn, w1, b1 = (dev(a, torch.float32) for a in (1 + 0.2 * normal(rng, 4, C), normal(rng, 4 * C, C) / 6, normal(rng, 4 * C)))
    w2 = dev(normal(rng, C, 4 * C) / 11, torch.float32)
    agg = emp.mp_forward(model, g, 0, sp, x)
    X, A, N = host(x).reshape(-1, 16 * C), host(agg).reshape(-1, 16 * C), g.n_atoms
    ry, rs = orow.rms_norm(X, host(wn), A)
    if quantize:
        q, scale, s = emp.mp_rms_norm(agg, wn, residual=x, quantize=True)
        wq, ws = to_e4m3(host(w1))
        h = emp.mp_dense(q[:, 0, :], wq, b1, activation="silu", x_scale=scale, w_scale=ws, out_dtype=torch.float32)
        rh = orow.dense(host(q)[:, 0, :] * host(scale)[:, None], host(wq) * host(ws)[:, None], host(b1), "silu")[0]
        assert np.abs(host(h) - rh).max() <= 1e-5 * np.abs(rh).max()
        assert np.abs(host(h) - orow.dense(ry[:, :C], host(w1), host(b1), "silu")[0]).max() <= 0.1 * np.abs(rh).max()
        return
    y, s = emp.mp_rms_norm(agg, wn, residual=x)
    h, z = emp.mp_dense(y[:, 0, :], w1, b1, activation="silu", keep_z=True)
    out = emp.mp_dense(h, w2, residual=s[:, 0, :])
    rh, rz = orow.dense(ry[:, :C], host(w1), host(b1), "silu")
    rout = orow.dense(rh, host(w2), residual=rs[:, :C])[0]
    assert np.abs(host(out) - rout).max() <= 1e-5 * np.abs(rout).max()
    assert torch.isfinite(emp.mp_forward(model, g, 1, sp, s)).all()
    # the block's gradient for dE/dout = go, dE/ds = go on degree 0 and zero elsewhere
    go = dev(normal(rng, N, C), torch.float32)
    g_h, g_w2, _ = emp.mp_dense_grad(go, h, w2)
    g_y0, g_w1, g_b1 = emp.mp_dense_grad(g_h, y[:, 0, :], w1, z=z, activation="silu")
    gy, gs = torch.zeros_like(y), torch.zeros_like(y)
    gy[:, 0], gs[:, 0] = g_y0, go
    g_x, g_wn = emp.mp_rms_norm_grad(gy, s, wn, g_s=gs)
    r_h, r_w2, _ = orow.dense_grad(host(go), rh, host(w2))
    r_y0, r_w1, r_b1 = orow.dense_grad(r_h, ry[:, :C], host(w1), rz, "silu")
    pad = lambda a: np.concatenate([a, np.zeros((N, 15 * C))], 1)  # noqa: E731
    r_x, r_wn = orow.rms_norm_grad(pad(r_y0), rs, host(wn), pad(host(go)))
    for got, ref in ((g_h, r_h), (g_w2, r_w2), (g_w1, r_w1), (g_b1, r_b1), (g_x, r_x), (g_wn, r_wn)):
        assert np.abs(host(got).reshape(ref.shape) - ref).max() <= 2e-5 * np.abs(ref).max()
    assert emp.last_device_error() == 0


# ------------------------------------------------------------------ refusals that need tensors on the device
def test_refusals():
    x, w = torch.zeros((4, 32), device="cuda"), torch.zeros((8, 32), device="cuda")
    h = x.bfloat16()
    z = torch.zeros((4, 8), device="cuda")
    bad = [lambda: emp.mp_rms_norm(x.cpu()), lambda: emp.mp_rms_norm(x.double()), lambda: emp.mp_rms_norm(x, eps=0.0),
           lambda: emp.mp_rms_norm(x, eps=float("nan")), lambda: emp.mp_rms_norm(x, residual=h),
           lambda: emp.mp_rms_norm(x, residual=x[:3]), lambda: emp.mp_rms_norm(x, x[0, :31]),
           lambda: emp.mp_rms_norm(x, torch.zeros((4, 3), device="cuda")), lambda: emp.mp_rms_norm(x, h[0]),
           lambda: emp.mp_rms_norm(torch.zeros((1, 8193), device="cuda")), lambda: emp.mp_rms_norm(x[:, :0]),
           lambda: emp.mp_rms_norm_grad(x[:3], x), lambda: emp.mp_rms_norm_grad(h, x),
           lambda: emp.mp_dense(x, w[:, :31]), lambda: emp.mp_dense(x, w.bfloat16()), lambda: emp.mp_dense(x, w, x[0]),
           lambda: emp.mp_dense(x, w, activation="tanh"), lambda: emp.mp_dense(x, w, residual=x),
           lambda: emp.mp_dense(x, w, out_dtype=torch.bfloat16), lambda: emp.mp_dense(x, w.cpu()),
           lambda: emp.mp_dense(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)),
           lambda: emp.mp_dense(x, w, x_scale=x[:, 0], w_scale=w[:, 0]),
           lambda: emp.mp_dense(x.to(torch.float8_e5m2), w.to(torch.float8_e5m2)),
           lambda: emp.mp_dense_grad(z, x, w, activation="silu"), lambda: emp.mp_dense_grad(z, x, w, z=z),
           lambda: emp.mp_dense_grad(z[:3], x, w), lambda: emp.mp_dense_grad(z.half(), x, w)]
    for i, f in enumerate(bad):
        with pytest.raises(emp.EmpError):
            f()
            pytest.fail(f"call {i} was accepted")
    a = emp.DenseGradC(700, 64, 64, 0, 0, *([x.data_ptr(), 64, None, 0] + [x.data_ptr(), 64] * 2), x.data_ptr(), 64,
                       x.data_ptr(), x.data_ptr())
    need = emp.lib().mp_dense_grad_workspace_bytes(ctypes.byref(a))
    assert need > 0
    assert emp.lib().mp_dense_grad(ctypes.byref(a), x.data_ptr() // 256 * 256, need - 1, None) == -6


# ------------------------------------------------------------------ alignments
@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 5), (3000, 31), (70, 77), (40, 515), (9, 1453), (4, 4097), (3, 8191), (700, 64)])
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 0), (0, 3), (3, 5)])
def test_norm_of_any_alignment(rows, cols, off, pad, type):
    """Rows `off` elements past a 16-byte boundary and `pad` elements apart; the residual aligned otherwise."""
    t, rng = TYPES[type], np.random.default_rng(rows + cols + off)

    def view(a, off, pad):
        full = torch.zeros(rows * (cols + pad) + off, dtype=t, device="cuda")
        v = torch.as_strided(full, (rows, cols), (cols + pad, 1), off)
        v.copy_(dev(a, t))
        return v

    x, r, g = (view(normal(rng, rows, cols), o, p) for o, p in ((off, pad), (pad, off), (off, 0)))
    w = dev(1 + 0.3 * normal(rng, cols), t)
    y, s = emp.mp_rms_norm(x, w, residual=r, eps=EPS)
    ry, rs = orow.rms_norm(host(x), host(w), host(r), EPS)
    near(y, ry, (half_step(t) + 32 * U) * np.abs(ry) + floor_of(t), "y")
    near(s, rs, (half_step(t) + U) * np.abs(rs) + floor_of(t), "s")
    q, scale, s2 = emp.mp_rms_norm(x, w, residual=r, eps=EPS, quantize=True)
    assert torch.equal(s, s2)
    rscale = orow.scale_of(ry)
    near(scale, rscale, 40 * U * rscale, "scale")
    value = host(q) * host(scale)[:, None]
    assert np.all(np.abs(value - ry) <= np.maximum(2.0 ** -4 * np.abs(ry), 2.0 ** -10 * rscale[:, None]) + 64 * U * np.abs(ry))
    S, G, W = host(x), host(g), host(w)
    g_x, g_w = emp.mp_rms_norm_grad(g, x, w, g_s=r, eps=EPS)
    rx, rw = orow.rms_norm_grad(G, S, W, host(r), EPS)
    rstd = 1 / np.sqrt((S * S).mean(1, keepdims=True) + EPS)
    n, h = S * rstd, G * W
    size = rstd * (np.abs(h) + np.abs(n) * np.abs(h * n).mean(1, keepdims=True)) + np.abs(host(r))
    near(g_x, rx, half_step(t) * np.abs(rx) + 64 * U * size + floor_of(t), "g_x")
    near(g_w, rw, half_step(t) * np.abs(rw) + (rows / 592 + 400) * U * np.abs(G * n).sum(0) + floor_of(t), "g_w")


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows", [3, 150])
@pytest.mark.parametrize("off,pad", [(1, 0), (0, 3), (2, 2)])
def test_dense_of_any_alignment(rows, off, pad, type):
    """x, W, the residual and g off 16-byte boundaries, outputs of rows that are off them too."""
    t, rng = TYPES[type], np.random.default_rng(rows + off)
    K, N = 70, 45

    def view(a):
        full = torch.zeros(a.shape[0] * (a.shape[1] + pad) + off, dtype=t, device="cuda")
        v = torch.as_strided(full, a.shape, (a.shape[1] + pad, 1), off)
        v.copy_(dev(a, t))
        return v

    x, w, r, g, z0 = (view(a) for a in (normal(rng, rows, K), normal(rng, N, K) / 8, normal(rng, rows, N), normal(rng, rows, N),
                                        normal(rng, rows, N)))
    y, z = emp.mp_dense(x, w, activation="gelu", residual=r, keep_z=True)
    ry, rz, ty, tz = dense_tol(host(x), host(w), None, host(r), "gelu", t, K)
    near(z, rz, tz, "z")
    near(y, ry, ty, "y")
    got = emp.mp_dense_grad(g, x, w, z=z0, activation="silu")
    ref = emp.mp_dense_grad(*(a.contiguous().clone() for a in (g, x, w)), z=z0.contiguous().clone(), activation="silu")
    for a, b in zip(got, ref):
        assert (a.double() - b.double()).abs().max() <= (4 * half_step(t) + 1e-5) * b.double().abs().max()


# ------------------------------------------------------------------ the ends of the range
EXTREME = [0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 3.0, -3.0, 8.0, -8.0, 20.0, -20.0, 42.9, -42.9, 43.1, -43.1, 88.0, -88.0, 95.0, -95.0,
           1e4, -1e4, 1e10, -1e10, 1e30, -1e30]


@pytest.mark.parametrize("rows", [16, 160])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_over_the_whole_range(act, rows):
    """y and dE/dx of a one-to-one layer (x 1, weights 1): z is x to 2^-20.  SiLU and GELU with 32 u |z| (the exponential's
    argument and the approximation of the normal distribution, 1.5e-7 / 2, included) and 2^-20 |z| times a slope below
    1.13; their slopes likewise with 64 u (1 + |z|) below |z| = 20, and exact limits beyond."""
    z = np.array((EXTREME * 7)[:rows]).reshape(rows, 1)
    x, w = dev(z, torch.float32), torch.ones((20, 1), device="cuda")
    z = host(x)
    y = host(emp.mp_dense(x, w, activation=act))
    with np.errstate(over="ignore"):
        ref, slope = orow.activation(z, act), orow.slope(z, act)
    assert np.all(np.isfinite(y)) and np.all(np.abs(y - ref) <= (32 * U + 1.13 * 2.0 ** -20) * np.abs(z) + 1e-37)
    assert np.all(y[z[:, 0] < -100] == 0)
    g = torch.ones((rows, 20), device="cuda")
    g_x, _, g_b = emp.mp_dense_grad(g, x, w, z=x.expand(rows, 20).contiguous(), activation=act)
    near = np.abs(z[:, 0]) <= 20
    d = np.abs(host(g_x) / 20 - slope)[:, 0]
    assert np.all(d[near] <= 64 * U * (1 + np.abs(z[near, 0])) + 2.0 ** -20 * 20) and np.all(d[~near] <= 2.0 ** -19)
    assert torch.isfinite(g_b).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_non_finite_values_through_an_activation(act):
    """+inf stays, -inf and NaN give NaN as z sigma(z) and z Phi(z) do, and the neighbouring columns are not touched."""
    x = torch.tensor([[float("inf")], [float("-inf")], [float("nan")], [1.0]], device="cuda").repeat(10, 1)
    w = torch.zeros((40, 1), device="cuda", dtype=torch.float32)
    w[7], w[20] = 1.0, 1.0
    for rows in (8, 40):
        for t in (torch.bfloat16, torch.float16):
            y = emp.mp_dense(x[:rows].to(t), w.to(t), residual=torch.ones((rows, 40), device="cuda", dtype=t), activation=act)
            col = y[:, 7].float()
            assert torch.isinf(col[0::4]).all() and torch.isnan(col[1::4]).all() and torch.isnan(col[2::4]).all()
            assert torch.isfinite(col[3::4]).all() and torch.equal(y[3::4, 0], torch.ones_like(y[3::4, 0]))


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows come out as they do alone."""
    rows, n = 1_100_000, 300
    t = torch.bfloat16
    w, wn = torch.randn((2048, 32), device="cuda").to(t), torch.ones(2048, device="cuda", dtype=t)
    x = torch.randn((rows, 32), device="cuda").to(t)
    y, z = emp.mp_dense(x, w, activation="silu", keep_z=True)
    ys, zs = emp.mp_dense(x[-n:], w, activation="silu", keep_z=True)
    assert torch.equal(y[-n:], ys) and torch.equal(z[-n:], zs)
    # the 300 rows alone split their 2048 products (too few tiles for the SMs), the many rows do not: the two sums are each
    # within 2 (n + 8) u sum|terms| of the exact one before they are rounded by at most half a step each
    g_x, _, _ = emp.mp_dense_grad(y, x, w, z=z, activation="silu", need_weight=False, need_bias=False)
    alone = emp.mp_dense_grad(ys, x[-n:], w, z=zs, activation="silu")[0]
    size = (ys.double() * 1.13).abs() @ w.double().abs()
    top = torch.maximum(g_x[-n:].double().abs(), alone.double().abs())
    assert torch.all((g_x[-n:].double() - alone.double()).abs() <= 2 * half_step(t) * top + 4 * (2048 + 8) * U * size)
    v, s = emp.mp_rms_norm(y, wn, residual=z)
    vs, ss = emp.mp_rms_norm(ys, wn, residual=zs)
    assert torch.equal(v[-n:], vs) and torch.equal(s[-n:], ss)
    q, scale, _ = emp.mp_rms_norm(y, wn, quantize=True)
    qs, scales, _ = emp.mp_rms_norm(ys, wn, quantize=True)
    assert torch.equal(q[-n:].view(torch.uint8), qs.view(torch.uint8)) and torch.equal(scale[-n:], scales)
    g_x, _ = emp.mp_rms_norm_grad(v, s, wn, g_s=z)
    assert torch.equal(g_x[-n:], emp.mp_rms_norm_grad(vs, ss, wn, g_s=zs)[0])
    del y, z, v, s, q, g_x
    odd = torch.randn((rows, 1999), device="cuda", dtype=t)
    v, _ = emp.mp_rms_norm(odd, wn[:1999])
    vs, _ = emp.mp_rms_norm(odd[-n:].clone(), wn[:1999])
    assert (v[-n:].float() - vs.float()).abs().max() <= 2.0 ** -7 * vs.float().abs().max()


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_a_weight_gradient_over_many_rows(type):
    """300000 rows: the sum of 300000 products keeps 2^-17 of its scale in FP32 and half a step in bf16 (2-norm)."""
    t, rng = TYPES[type], np.random.default_rng(23)
    x, g = dev(normal(rng, 300000, 64), t), dev(normal(rng, 300000, 48), t)
    _, g_w, g_b = emp.mp_dense_grad(g, x, torch.zeros((48, 64), device="cuda", dtype=t), need_x=False)
    ref = g.double().t() @ x.double()
    assert ((g_w.double() - ref).norm() / ref.norm()).item() <= (2.0 ** -17 if t == torch.float32 else half_step(t))
    assert ((g_b.double() - g.double().sum(0)).norm() / g.double().sum(0).norm()).item() <= (2.0 ** -17 if t == torch.float32 else half_step(t))


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 3), (2, 1023), (15, 66), (33, 515), (2401, 65), (20003, 34), (9999, 129), (700, 2047)])
def test_norm_of_contiguous_rows_off_16_bytes(rows, cols, type):
    """Rows that begin and end inside a 16-byte vector or a 32-bit word, with and without a residual, weights and 8-bit
    values, forward and back; what lies behind the last row stays.  Tolerances as in the tests above."""
    t, rng = TYPES[type], np.random.default_rng(rows * 31 + cols)
    x, r, g = (dev(normal(rng, rows, cols), t) for _ in range(3))
    w = dev(1 + 0.3 * normal(rng, cols), t)
    for res in (None, r):
        for weight in (None, w):
            ry, rs = orow.rms_norm(host(x), host(weight), host(res), EPS)
            y, s = emp.mp_rms_norm(x, weight, residual=res, eps=EPS)
            near(y, ry, (half_step(t) + 32 * U) * np.abs(ry) + floor_of(t), "y")
            near(s, rs, (half_step(t) + U) * np.abs(rs) + floor_of(t), "s")
            q, scale, s2 = emp.mp_rms_norm(x, weight, residual=res, eps=EPS, quantize=True)
            rscale = orow.scale_of(ry)
            near(scale, rscale, 40 * U * rscale, "scale")
            value = host(q) * host(scale)[:, None]
            assert torch.equal(s, s2)
            assert np.all(np.abs(value - ry) <= np.maximum(2.0 ** -4 * np.abs(ry), 2.0 ** -10 * rscale[:, None]) + 64 * U * np.abs(ry))
    S, G, W = host(x), host(g), host(w)
    rstd = 1 / np.sqrt((S * S).mean(1, keepdims=True) + EPS)
    n, h = S * rstd, G * W
    for through in (None, r):
        g_x, g_w = emp.mp_rms_norm_grad(g, x, w, g_s=through, eps=EPS)
        rx, rw = orow.rms_norm_grad(G, S, W, host(through), EPS)
        size = rstd * (np.abs(h) + np.abs(n) * np.abs(h * n).mean(1, keepdims=True)) + (0 if through is None else np.abs(host(through)))
        near(g_x, rx, half_step(t) * np.abs(rx) + 64 * U * size + floor_of(t), "g_x")
        near(g_w, rw, half_step(t) * np.abs(rw) + (rows / 592 + 400) * U * np.abs(G * n).sum(0) + floor_of(t), "g_w")
    # the library writes rows it was given and nothing behind them
    code = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[t]
    for y_code, y_type in ((code, t), (3, torch.uint8)):
        y = torch.full(((rows + 2) * cols,), 7, dtype=y_type, device="cuda")
        sums = torch.full(((rows + 2) * cols,), 7, dtype=t, device="cuda")
        scale = torch.full((rows + 1,), 7.0, device="cuda")
        a = emp.RmsNormC(rows, cols, code, y_code, 0, EPS, x.data_ptr(), cols, r.data_ptr(), cols, w.data_ptr(), y.data_ptr(), cols,
                         scale.data_ptr() if y_code == 3 else None, sums.data_ptr(), cols)
        assert emp.lib().mp_rms_norm(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
        assert torch.all(y[rows * cols:].float() == 7) and torch.all(sums[rows * cols:].float() == 7) and scale[rows] == 7


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("K,N", [(64, 128), (96, 72), (40, 260), (33, 45)])
@pytest.mark.parametrize("residual,keep", [(False, False), (True, False), (True, True)])
def test_dense_of_many_tiles_per_block(K, N, residual, keep, type):
    """More than two tiles of 128 rows for every SM, the last one ragged: what the epilogue asks for ahead of a tile belongs to it."""
    t, rows = TYPES[type], 2 * 148 * 128 + 19000 + 77
    rng = np.random.default_rng(K + N)
    x, w, b = dev(normal(rng, rows, K), t), dev(normal(rng, N, K) / np.sqrt(K), t), dev(normal(rng, N), t)
    r = dev(normal(rng, rows, N), t) if residual else None
    out = emp.mp_dense(x, w, b, activation="silu", residual=r, keep_z=keep)
    y, z = out if keep else (out, None)
    ry, rz, ty, tz = dense_tol(host(x), host(w), host(b), host(r), "silu", t, K)
    near(y, ry, ty, "y")
    if keep:
        near(z, rz, tz, "z")


@pytest.mark.parametrize("type", [*TYPES, "e4m3"])
@pytest.mark.parametrize("rows,K,N", [(12, 2001, 99), (16, 1025, 33), (1, 1153, 130), (9, 2047, 7)])
def test_dense_of_few_rows_off_16_bytes(rows, K, N, type):
    """Rows of a k that is odd and longer than what is staged at once."""
    rng = np.random.default_rng(rows * K + N)
    x, w, r = normal(rng, rows, K), normal(rng, N, K) / np.sqrt(K), normal(rng, rows, N)
    if type == "e4m3":
        t = torch.float16
        (x, xs), (w, ws) = to_e4m3(x), to_e4m3(w)
        r = dev(r, t)
        y = emp.mp_dense(x, w, activation="silu", residual=r, x_scale=xs, w_scale=ws, out_dtype=t)
        X, W = host(x) * host(xs)[:, None], host(w) * host(ws)[:, None]
    else:
        t = TYPES[type]
        x, w, r = dev(x, t), dev(w, t), dev(r, t)
        y = emp.mp_dense(x, w, activation="silu", residual=r)
        X, W = host(x), host(w)
    ry, _, ty, _ = dense_tol(X, W, None, host(r), "silu", t, K)
    near(y, ry, ty, "y")
