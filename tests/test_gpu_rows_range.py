"""The row-wise operators over the rest of their range, against the float64 oracle: forms that take several tiles per
block, values at the ends of the types, long sums.  Tolerances as derived in test_gpu_rows.py where nothing else is said."""
import ctypes

import numpy as np
import pytest

from oracle import rows as orow
from test_gpu_rows import TYPES, U, dense_tol, dev, floor_of, half_step, host, near, normal, to_e4m3

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


# ------------------------------------------------------------------ activations, relative to their own size
def activation_tol(z, act, t):
    """Relative: GELU (32 + 1.5 z^2) u (2^x and 1/x 4 u each with what their arguments' errors do, the polynomial's fit 2 u and eight
    steps, three products; z^2 / 2 is rounded three times); SiLU 8 u (2^x 4 u, 1/x 2 u, the sum and the product) and
    |z| log 2 times two roundings of the exponent.  GELU of 16-bit types: a fit within 5e-5."""
    if act == "gelu":
        return (32 + 1.5 * z * z) * U + (5e-5 if t != torch.float32 else 0)
    return (8 + 2 * np.abs(z)) * U


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows", [8, 16, 200, 1620])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_keep_their_digits(act, rows, type):
    """z = x 1 with at most 8 bits of x, so z has no error; down to where the results leave the normal range."""
    t = TYPES[type]
    low = -12.5 if act == "gelu" else -80.0
    x = torch.linspace(low, -low, rows).to(torch.bfloat16).unsqueeze(1)
    z = x.double().numpy()
    w = torch.ones((12, 1), device="cuda", dtype=t)
    y = host(emp.mp_dense(x.cuda().to(t), w, activation=act))
    ref = orow.activation(z, act)
    near(torch.from_numpy(y), np.broadcast_to(ref, y.shape), (half_step(t) + activation_tol(z, act, t)) * np.abs(ref) + floor_of(t), act)
    # the slope, where its two terms do not cancel: through g_x = g act'(z) W with one column
    g = torch.ones((len(z), 1), device="cuda", dtype=t)
    g_x = host(emp.mp_dense_grad(g, x.cuda().to(t), w[:1], z=x.cuda().to(t), activation=act, need_weight=False)[0])
    if act == "gelu":
        size = orow.phi(z) + np.abs(z) * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    else:
        p = 1 / (1 + np.exp(-z))
        size = p + np.abs(z) * p * (1 - p)
    tol = (2 * half_step(t) + 2.0 ** -20) * np.abs(orow.slope(z, act)) + (activation_tol(z, act, t) + 8 * U) * size + 2 * floor_of(t)
    near(torch.from_numpy(g_x), orow.slope(z, act), tol, act + "'")


# ------------------------------------------------------------------ long sums of one sign
# The tensor cores' adder truncates: each of the n MMAs of a chain takes half a unit in the last place off the running sum on
# average, n / 4 of the last sum's units in all, a unit being 0.72 2^-23 on average: 2.15e-8 n, 8.8e-5 for the longest chain of 4096 MMAs.
CHAIN = 1e-4


def columns(rng, rows, cols, t, scale=1.0):
    """Positive values, every column of another size (else all outputs would be rounded alike)."""
    return dev(rng.uniform(0.5, 1.5, (rows, cols)) * rng.uniform(1, 2, (1, cols)) * scale, t)


def short_of(got, ref, t):
    """Every output within the chain's part and half a step; their mean within the chain's part and five deviations of the rounding."""
    d = got.double() / ref - 1
    e = half_step(t) if t != torch.float32 else U
    assert d.abs().max().item() <= CHAIN + e, d.abs().max().item()
    assert abs(d.mean().item()) <= CHAIN + 5 * e / np.sqrt(3 * d.numel()), d.mean().item()


@pytest.mark.parametrize("type", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [65536, 300000])
def test_a_weight_gradient_of_one_sign_over_many_rows(rows, type):
    t, rng = TYPES[type], np.random.default_rng(rows)
    x, g = columns(rng, rows, 64, t), columns(rng, rows, 48, t, 2.0 ** -6 if type == "f16" else 1.0)
    _, g_w, g_b = emp.mp_dense_grad(g, x, torch.zeros((48, 64), device="cuda", dtype=t), need_x=False)
    short_of(g_w, g.double().t() @ x.double(), t)
    short_of(g_b, g.double().sum(0), t)


@pytest.mark.parametrize("type", ["f32", "bf16", "f16", "e4m3"])
@pytest.mark.parametrize("rows", [40, 300])
def test_a_layer_of_one_sign_and_the_longest_k(rows, type):
    """e4m3 inputs with FP32 outputs show the chain (2048 MMAs of 32) without the output's rounding; FP32 inputs leave the chain
    every 96 of k and add 683 parts rounded to nearest (at most 683 u) to 36 MMAs' truncation."""
    K, N, rng = 65536, 64, np.random.default_rng(rows)
    if type == "e4m3":
        x, w = (dev(np.exp(rng.uniform(-4, 0, (n, K))), torch.float32).to(torch.float8_e4m3fn) for n in (rows, N))
        xs, ws = (dev(rng.uniform(1, 2, n), torch.float32) for n in (rows, N))
        y = emp.mp_dense(x, w, x_scale=xs, w_scale=ws, out_dtype=torch.float32)
        short_of(y, (x.double() * xs.double()[:, None]) @ (w.double() * ws.double()[:, None]).t(), torch.float32)
        return
    t = TYPES[type]
    x, w = (columns(rng, K, n, t, 1 / 64).t().contiguous() for n in (rows, N))
    y, ref = emp.mp_dense(x, w), x.double() @ w.double().t()
    if type == "f32":
        assert (y.double() / ref - 1).abs().max().item() <= (683 + 2 * 36) * U
    else:
        short_of(y, ref, t)


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("rows,K,N", [(17, 65536, 5), (40, 20000, 64), (128, 33000, 128), (33, 65536, 497), (1, 65536, 33)])
def test_scales_of_many_splits(rows, K, N, out):
    """A long k with few outputs is split, and the parts' sum still takes the scales."""
    t, rng = TYPES[out], np.random.default_rng(rows + K + N)
    (x, xs), (w, ws) = to_e4m3(normal(rng, rows, K) * np.exp(normal(rng, rows, 1))), to_e4m3(normal(rng, N, K) / np.sqrt(K))
    X, W = x.double() * xs.double()[:, None], w.double() * ws.double()[:, None]
    for act, bias in (("none", False), ("silu", True)):
        b = dev(normal(rng, N), torch.float32) if bias else None
        y = emp.mp_dense(x, w, b, activation=act, x_scale=xs, w_scale=ws, out_dtype=t)
        z = host(X @ W.t()) + (0 if b is None else host(b))
        ref = orow.activation(z, act)
        dz = (2.0 ** -20 + 2 * (K / 32 + 200) * U) * host(X.abs() @ W.abs().t()) + 8 * U * np.abs(z)    # an MMA sums 32 of k
        near(y, ref, half_step(t) * np.abs(ref) + 1.13 * dz + 16 * U * (np.abs(z) + np.abs(ref)) + floor_of(t), act)


# ------------------------------------------------------------------ infinite inputs, and values that become infinite
@pytest.mark.parametrize("rows,K,N", [(1, 64, 40), (8, 256, 100), (1, 4096, 40), (8, 2500, 100), (16, 2048, 2100), (40, 96, 33)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 3.4028e38])
def test_fp32_non_finite_inputs_of_few_rows(rows, K, N, value):
    """On SIMT and on the tensor cores: no other row or column changes, and a row of an infinite or NaN input has no
    finite output.  (3.4028e38 counts as infinite on the tensor cores alone: its outputs are right where they are finite.)"""
    rng = np.random.default_rng(rows + K)
    t = torch.float32
    x, w = dev(normal(rng, rows, K), t), dev(1 + 0.1 * normal(rng, N, K), t)
    clean = emp.mp_dense(x, w)
    xb = x.clone()
    xb[rows - 1, K // 2] = value
    bad = emp.mp_dense(xb, w)
    assert torch.equal(bad[:-1], clean[:-1])
    last = bad[-1].double()
    if np.isfinite(value):
        ref = xb[-1].double() @ w.double().t()
        ok = torch.isfinite(last)
        assert ((last - ref).abs() <= 1e-5 * ref.abs())[ok].all()
    else:
        assert not torch.isfinite(last).any()
    wb = w.clone()
    wb[N // 2, 1] = value
    bad = emp.mp_dense(x, wb)
    keep = torch.arange(N, device="cuda") != N // 2
    assert torch.equal(bad[:, keep], clean[:, keep])
    if not np.isfinite(value):
        assert not torch.isfinite(bad[:, N // 2]).any()


@pytest.mark.parametrize("rows,K,N", [(1, 64, 40), (8, 70, 33), (300, 64, 96)])
def test_fp32_gradient_of_non_finite_inputs(rows, K, N):
    rng = np.random.default_rng(rows + N)
    t = torch.float32
    x, w, g = dev(1 + 0.1 * normal(rng, rows, K), t), dev(1 + 0.1 * normal(rng, N, K), t), dev(normal(rng, rows, N), t)
    g_x, g_w, g_b = emp.mp_dense_grad(g, x, w)
    gb = g.clone()
    gb[rows - 1, N - 1] = float("inf")
    b_x, b_w, b_b = emp.mp_dense_grad(gb, x, w)
    assert torch.equal(b_x[:-1], g_x[:-1]) and not torch.isfinite(b_x[-1]).any()
    assert torch.equal(b_w[:-1], g_w[:-1]) and not torch.isfinite(b_w[-1]).any()
    assert torch.equal(b_b[:-1], g_b[:-1]) and torch.isinf(b_b[-1])


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -60, 2.0 ** -110])
@pytest.mark.parametrize("rows,K,N", [(8, 256, 100), (300, 64, 96), (300, 500, 96)])
def test_fp32_of_small_magnitudes(rows, K, N, scale):
    rng = np.random.default_rng(rows + K)
    t = torch.float32
    x, w = dev(normal(rng, rows, K) * scale, t), dev(normal(rng, N, K) * 2.0 ** 20, t)
    y, _, ty, _ = dense_tol(host(x), host(w), None, None, "none", t, K)
    near(emp.mp_dense(x, w), y, ty, "y")


@pytest.mark.parametrize("act,z0", [("silu", 2.4), ("gelu", 1.4142)])
def test_fp16_gradient_whose_product_with_the_slope_leaves_the_type(act, z0):
    """|g act'(z)| above 65504 is infinite as an operand in fp16: its row of g_x and its column's g_weight show it, no others do;
    below that, and in bf16, they are finite."""
    rng = np.random.default_rng(29)
    rows, K, N = 150, 64, 48
    for t, top, finite in ((torch.float16, 60000.0, False), (torch.float16, 57000.0, True), (torch.bfloat16, 60000.0, True)):
        x, w = dev(normal(rng, rows, K) / 64, t), dev(normal(rng, N, K) / 64, t)
        z, g = dev(normal(rng, rows, N), t), dev(normal(rng, rows, N), t)
        clean = emp.mp_dense_grad(g, x, w, z=z, activation=act)
        zb, gb = z.clone(), g.clone()
        zb[7, 5], gb[7, 5] = z0, top
        g_x, g_w, _ = emp.mp_dense_grad(gb, x, w, z=zb, activation=act)
        rest = torch.arange(rows, device="cuda") != 7
        cols = torch.arange(N, device="cuda") != 5
        assert torch.equal(g_x[rest], clean[0][rest])
        assert torch.isfinite(g_w[cols]).all()
        assert torch.isfinite(g_x[7]).all() == finite and torch.isfinite(g_w[5]).all() == finite
        if not finite:
            assert not torch.isfinite(g_x[7]).any() and not torch.isfinite(g_w[5]).any()


# ------------------------------------------------------------------ what lies beside an output
def framed(rows, cols, pitch, t):
    """A buffer of sentinels and the view of rows inside it, both of whose ends it goes beyond by 64 elements."""
    full = torch.full((rows * pitch + 128,), -77.0, dtype=t, device="cuda")
    return full, torch.as_strided(full, (rows, cols), (pitch, 1), 64)


def only_inside(full, inner):
    got = inner.clone()
    inner.fill_(-77.0)
    assert torch.all(full == -77.0)
    return got


@pytest.mark.parametrize("type", list(TYPES))
@pytest.mark.parametrize("rows,K,N", [(1, 2500, 1), (1, 2500, 37), (40, 96, 1), (40, 96, 13), (40, 200, 37), (300, 64, 61), (300, 500, 7)])
def test_aligned_pitches_of_odd_widths(rows, K, N, type):
    """Rows of y, z and g_x that begin on 16 bytes and end inside them, single rows, and weight gradients of such a width: the
    bytes behind a row's last element and behind the last row stay."""
    t, rng = TYPES[type], np.random.default_rng(rows + K + N)
    code, L, st = {"f32": 0, "bf16": 1, "f16": 2}[type], emp.lib(), torch.cuda.current_stream().cuda_stream
    x, w, b = dev(normal(rng, rows, K), t), dev(normal(rng, N, K) / np.sqrt(K), t), dev(normal(rng, N), t)
    pitch = -(-N // 16) * 16 + 16
    r = framed(rows, N, pitch, t)[1]
    r.copy_(dev(normal(rng, rows, N), t))
    (yf, y), (zf, z) = framed(rows, N, pitch, t), framed(rows, N, pitch, t)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    a = emp.DenseC(rows, K, N, code, code, 1, x.data_ptr(), K, None, w.data_ptr(), K, None, b.data_ptr(), r.data_ptr(), pitch, y.data_ptr(),
                   pitch, z.data_ptr(), pitch)
    assert L.mp_dense(ctypes.byref(a), ws.data_ptr(), ws.numel(), st) == 0
    ry, rz, ty, tz = dense_tol(host(x), host(w), host(b), host(r), "silu", t, K)
    near(only_inside(yf, y), ry, ty, "y")
    near(only_inside(zf, z), rz, tz, "z")
    # the other way about: g_x of width N from N columns of a weight, its gradient [K][N] and a bias gradient of K
    g, v, xn = dev(normal(rng, rows, K), t), dev(normal(rng, K, N) / np.sqrt(K), t), dev(normal(rng, rows, N), t)
    (xf, gx), (wf, gw), (bf, gb) = framed(rows, N, pitch, t), framed(K, N, N, t), framed(1, K, K, t)
    d = emp.DenseGradC(rows, N, K, code, 0, g.data_ptr(), K, None, 0, xn.data_ptr(), N, v.data_ptr(), N, gx.data_ptr(), pitch, gw.data_ptr(),
                       gb.data_ptr())
    assert L.mp_dense_grad(ctypes.byref(d), ws.data_ptr(), ws.numel(), st) == 0
    rx, rw, rb = orow.dense_grad(host(g), host(xn), host(v))
    tol = lambda ref, S, n: half_step(t) * np.abs(ref) + (2.0 ** -20 + 2 * (n + 8) * U) * S + floor_of(t)  # noqa: E731
    G = np.abs(host(g))
    near(only_inside(xf, gx), rx, tol(rx, G @ np.abs(host(v)), K), "g_x")
    near(only_inside(wf, gw), rw, tol(rw, G.T @ np.abs(host(xn)), rows), "g_w")
    near(only_inside(bf, gb), rb[None], tol(rb, G.sum(0), rows)[None], "g_b")
    # one output, whose weight gradient is a single row of K
    g1, (of, o) = dev(normal(rng, rows, 1), t), framed(1, K - 3, K - 3, t)
    d = emp.DenseGradC(rows, K - 3, 1, code, 0, g1.data_ptr(), 1, None, 0, x.data_ptr(), K, None, 0, None, 0, o.data_ptr(), None)
    assert L.mp_dense_grad(ctypes.byref(d), ws.data_ptr(), ws.numel(), st) == 0
    X = host(x)[:, :K - 3]
    near(only_inside(of, o), host(g1).T @ X, tol(host(g1).T @ X, np.abs(host(g1)).T @ np.abs(X), rows), "g_w of one output")


@pytest.mark.parametrize("rows,K,N", [(5, 64, 40), (16, 2100, 33), (200, 128, 96), (300, 100, 61)])
def test_nan_of_8_bits_stays_in_its_row_and_column(rows, K, N):
    rng = np.random.default_rng(rows)
    (x, xs), (w, ws) = to_e4m3(normal(rng, rows, K)), to_e4m3(normal(rng, N, K))
    call = lambda a, b, c, d: emp.mp_dense(a, b, x_scale=c, w_scale=d, out_dtype=torch.float16)  # noqa: E731
    clean = call(x, w, xs, ws)
    xb, wb, sb = x.clone(), w.clone(), xs.clone()
    xb.view(torch.uint8)[1, 3], wb.view(torch.uint8)[N - 1, 0], sb[0] = 0x7f, 0xff, float("nan")
    bad = call(xb, wb, sb, ws)
    assert torch.isnan(bad[:2]).all() and torch.isnan(bad[:, -1]).all()
    assert torch.equal(bad[2:, :-1], clean[2:, :-1])
