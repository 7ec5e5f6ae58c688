"""The node-wise operators of the message-passing layers, as they are timed and compared.

Four operators, all on rows (one row per atom or per edge):

* ``norm``        s = x + residual, y = s / sqrt(mean(s^2) + eps) * w; y in the input's type, or in
                  8 bits (e4m3) with one scale per row.  With ``degrees`` the row is an atom's
                  [16, C] features and w is [4, C], one weight per degree and channel.
* ``norm_grad``   its gradient: g_x (which is the residual's too) and g_w.
* ``dense``       y = act(x W^T + b) + residual, inputs of 32, 16 or 8 bits (e4m3 with a scale per
                  row of x and of W), optionally with z = x W^T + b kept for the backward.
* ``dense_grad``  its gradient: g_x, g_W, g_b.

Plain torch operations where ``own`` is false, the library's entry points where it is true.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
EPS = 1e-6
E4M3_MAX = 448.0
TINY = 2.0 ** -110          # a row of y whose largest magnitude is below this has the scale 1


def norm_case(name, rows, cols, type, degrees=False, residual=True, quantize=False, spread=1):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "type": type, "degrees": degrees,
            "residual": residual, "quantize": quantize, "spread": spread}


def norm_grad_case(name, rows, cols, type, degrees=False, through=True):
    return {"name": name, "op": "norm_grad", "rows": rows, "cols": cols, "type": type, "degrees": degrees,
            "through": through}


def dense_case(name, rows, fan_in, fan_out, type, act="none", bias=True, residual=False, keep_z=False, spread=1):
    return {"name": name, "op": "dense", "rows": rows, "fan_in": fan_in, "fan_out": fan_out, "type": type, "act": act,
            "bias": bias, "residual": residual, "keep_z": keep_z, "spread": spread}


def dense_grad_case(name, rows, fan_in, fan_out, type, act="none"):
    return {"name": name, "op": "dense_grad", "rows": rows, "fan_in": fan_in, "fan_out": fan_out, "type": type,
            "act": act}


def listed():
    return [
        # the 64-atom cell with C = 64 channels: one layer's update and norm, where latency counts
        norm_case("norm_f32_n64", 64, 16 * 64, "f32", degrees=True),
        # the 4096-atom frame with C = 128: the update x + agg between two layers and its norm
        norm_case("norm_f32_n4096", 4096, 16 * 128, "f32", degrees=True),
        # per-edge features of the 512-atom frame at a width that no vector load divides
        norm_case("norm_bf16_edges_odd", 80896, 515, "bf16", residual=False),
        # screening in 8 bits: node rows of several frames normed straight into the product's operand
        norm_case("norm_bf16_to_e4m3", 16384, 16 * 128, "bf16", degrees=True, quantize=True),
        # training at the 4096-atom frame
        norm_grad_case("norm_grad_f32_n4096", 4096, 16 * 128, "f32", degrees=True),
        # training on per-edge rows in 16 bits
        norm_grad_case("norm_grad_bf16_edges", 80896, 512, "bf16"),
        # the degree-0 channels of eight atoms (a cluster around a defect): latency
        dense_case("dense_f32_few", 8, 256, 1024, "f32", act="silu", residual=True, spread=16),
        # a radial head over every edge of the 4096-atom frame, 64 -> 4 x 128
        dense_case("dense_f32_edges", 647168, 64, 512, "f32", act="silu"),
        # odd sizes in 16 bits, a training forward (z kept)
        dense_case("dense_bf16_odd", 20011, 515, 250, "bf16", act="gelu", residual=True, keep_z=True),
        # screening in 8 bits: full node rows of sixteen 4096-atom frames, 16 x 128 -> 512
        dense_case("dense_e4m3_nodes", 65536, 2048, 512, "e4m3", act="silu", residual=True),
        # training a radial head on the 512-atom frame's edges, FP32
        dense_grad_case("dense_grad_f32_edges", 80896, 128, 512, "f32", act="silu"),
        # training a wide node layer in 16 bits
        dense_grad_case("dense_grad_bf16_wide", 16384, 1024, 1024, "bf16", act="silu"),
    ]


def cost(case):
    """Roughly the plain form's seconds: its float products and its passes over memory."""
    w = work(case)
    return w["flops"] / 5e13 + 4 * w["bytes"] / 5e12


def log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    most = max(cost(c) for c in listed())
    while True:
        op = rng.choice(["norm", "norm", "norm_grad", "dense", "dense", "dense", "dense_grad", "dense_grad"])
        if op in ("norm", "norm_grad"):
            degrees = rng.random() < 0.5
            cols = 16 * 32 * rng.randint(1, 8) if degrees else log_int(rng, 8, 4096)
            rows, type = log_int(rng, 1, 200000), rng.choice(["f32", "bf16", "f16"])
            if op == "norm":
                case = norm_case("", rows, cols, type, degrees, rng.random() < 0.7, rng.random() < 0.35,
                                 rng.choice([1, 1, 2]))
            else:
                case = norm_grad_case("", rows, cols, type, degrees, rng.random() < 0.6)
        else:
            rows, fan_in, fan_out = log_int(rng, 1, 650000), log_int(rng, 8, 2048), log_int(rng, 1, 2048)
            if rng.random() < 0.5:                          # channel counts as the models have them
                fan_in, fan_out = -(-fan_in // 32) * 32, -(-fan_out // 32) * 32
            act = rng.choice(["none", "silu", "silu", "gelu"])
            if op == "dense":
                case = dense_case("", rows, fan_in, fan_out, rng.choice(["f32", "f32", "bf16", "f16", "e4m3"]), act,
                                  rng.random() < 0.7, rng.random() < 0.4, rng.random() < 0.3,
                                  rng.choice([1, 1, 1, 16]) if rows * fan_in < 2e7 else 1)
            else:
                case = dense_grad_case("", min(rows, 160000), fan_in, fan_out, rng.choice(["f32", "bf16", "f16"]), act)
        if 2e5 < work(case)["bytes"] and cost(case) <= most:
            return case


# ------------------------------------------------------------------ inputs
def rows_of(g, rows, cols, type, spread=1):
    """Normal rows of unequal sizes; spread > 1: every row is the start of one `spread` times as long."""
    wide = torch.randn((rows, spread * cols), device="cuda", generator=g)
    wide *= torch.exp(0.5 * torch.randn((rows, 1), device="cuda", generator=g))
    return wide.to(TYPES[type])[:, :cols]


def in_e4m3(a):
    """Rows in 8 bits and their scales."""
    scale = a.abs().amax(1) / E4M3_MAX
    return (a / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = case["type"]

    def normal(*shape, scale=1.0, type=t):
        return (scale * torch.randn(shape, device="cuda", generator=g)).to(TYPES[type])

    st = {"case": case}
    if case["op"] in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        w_shape = (4, cols // 16) if case["degrees"] else (cols,)
        st["w"] = (1.0 + 0.2 * torch.randn(w_shape, device="cuda", generator=g)).to(TYPES[t])
        # the degree of each of the 16 components, for the plain form
        st["degree"] = torch.tensor([0] + [1] * 3 + [2] * 5 + [3] * 7, device="cuda") if case["degrees"] else None
        x = rows_of(g, rows, cols, t, case.get("spread", 1))
        if case["op"] == "norm":
            st["x"] = x
            st["residual"] = normal(rows, cols) if case["residual"] else None
        else:
            st["s"], st["g"] = x, normal(rows, cols)
            st["g_s"] = normal(rows, cols) if case["through"] else None
        return st
    rows, fan_in, fan_out = case["rows"], case["fan_in"], case["fan_out"]
    weight = torch.randn((fan_out, fan_in), device="cuda", generator=g) / math.sqrt(fan_in)
    if case["op"] == "dense":
        out = "bf16" if t == "e4m3" else t
        x = rows_of(g, rows, fan_in, "f32" if t == "e4m3" else t, case["spread"])
        st["x"], st["x_scale"], st["w"], st["w_scale"] = x, None, weight.to(TYPES[out]), None
        if t == "e4m3":
            st["x"], st["x_scale"] = in_e4m3(x)
            st["w"], st["w_scale"] = in_e4m3(weight)
        st["b"] = normal(fan_out, scale=0.3, type="f32" if t == "e4m3" else t) if case["bias"] else None
        st["residual"] = normal(rows, fan_out, type=out) if case["residual"] else None
        return st
    st["x"], st["w"] = rows_of(g, rows, fan_in, t), weight.to(TYPES[t])
    st["g"] = normal(rows, fan_out)
    st["z"] = normal(rows, fan_out) if case["act"] != "none" else None
    return st


# ------------------------------------------------------------------ the plain forms
def per_column(st):
    """The weights of a row's columns: [4, C] ones, per degree and channel, spread over 16 C."""
    return st["w"].float() if st["degree"] is None else st["w"].float()[st["degree"]].flatten()


def plain_norm(st):
    case = st["case"]
    s = st["x"].float()
    if st["residual"] is not None:
        s = s + st["residual"].float()
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * per_column(st)
    out = TYPES[case["type"]]
    s = st["x"] if st["residual"] is None else s.to(out)
    if not case["quantize"]:
        return y.to(out), s
    amax = y.abs().amax(1)
    scale = torch.where(amax < TINY, torch.ones_like(amax), amax / E4M3_MAX)
    return (y / scale[:, None]).to(torch.float8_e4m3fn), scale, s


def plain_norm_grad(st):
    case = st["case"]
    s, g = st["s"].float(), st["g"].float()
    rstd = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS)
    n = s * rstd
    gw = g * per_column(st)
    g_x = rstd * (gw - n * (gw * n).mean(1, keepdim=True))
    if st["g_s"] is not None:
        g_x = g_x + st["g_s"].float()
    g_w = (g * n).sum(0, dtype=torch.float64)
    if case["degrees"]:
        g_w = torch.zeros(st["w"].shape, dtype=torch.float64, device=g_w.device).index_add_(
            0, st["degree"], g_w.view(16, -1))
    return g_x.to(TYPES[case["type"]]), g_w.to(TYPES[case["type"]])


def act_of(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def slope_of(z, act):
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


def plain_dense(st):
    case = st["case"]
    z = st["x"].float() @ st["w"].float().t()
    if st["x_scale"] is not None:
        z = z * st["x_scale"][:, None] * st["w_scale"]
    if st["b"] is not None:
        z = z + st["b"].float()
    y = act_of(z, case["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    out = torch.bfloat16 if case["type"] == "e4m3" else TYPES[case["type"]]
    return (y.to(out), z.to(out)) if case["keep_z"] else y.to(out)


def plain_dense_grad(st):
    case = st["case"]
    g = st["g"].float()
    if st["z"] is not None:
        g = g * slope_of(st["z"].float(), case["act"])
    out = TYPES[case["type"]]
    return (g @ st["w"].float()).to(out), (g.t() @ st["x"].float()).to(out), g.sum(0, dtype=torch.float64).to(out)


def run(st):
    case = st["case"]
    if own:
        import edge_message_passing_b200 as emp
        if case["op"] == "norm":
            return emp.mp_rms_norm(st["x"], st["w"], residual=st["residual"], eps=EPS, quantize=case["quantize"])
        if case["op"] == "norm_grad":
            return emp.mp_rms_norm_grad(st["g"], st["s"], st["w"], g_s=st["g_s"], eps=EPS)
        if case["op"] == "dense":
            return emp.mp_dense(st["x"], st["w"], st["b"], activation=case["act"], residual=st["residual"],
                                x_scale=st["x_scale"], w_scale=st["w_scale"], keep_z=case["keep_z"])
        return emp.mp_dense_grad(st["g"], st["x"], st["w"], z=st["z"], activation=case["act"])
    return {"norm": plain_norm, "norm_grad": plain_norm_grad, "dense": plain_dense,
            "dense_grad": plain_dense_grad}[case["op"]](st)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    b = SIZE[case["type"]]
    if case["op"] in ("norm", "norm_grad"):
        n = case["rows"] * case["cols"]
        weights = b * (case["cols"] // 4 if case["degrees"] else case["cols"])
        if case["op"] == "norm":
            out = n + 4 * case["rows"] if case["quantize"] else n * b
            sums = 2 * n * b if case["residual"] else 0           # the residual in, the sum out
            return {"bytes": n * b + sums + out + weights, "flops": 6 * n}
        return {"bytes": (3 + case["through"]) * n * b + 2 * weights, "flops": 12 * n}
    m, k, n = case["rows"], case["fan_in"], case["fan_out"]
    if case["op"] == "dense":
        o = 2 if case["type"] == "e4m3" else b
        scales = 4 * (m + n) if case["type"] == "e4m3" else 0
        bias = n * (4 if case["type"] == "e4m3" else b) if case["bias"] else 0
        return {"bytes": (m * k + n * k) * b + scales + bias + m * n * o * (1 + case["residual"] + case["keep_z"]),
                "flops": 2 * m * n * k}
    with_z = case["act"] != "none"
    return {"bytes": b * (m * n * (1 + with_z) + 2 * m * k + 2 * n * k + n), "flops": 4 * m * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits
def e4m3_values(v):
    """v (64 bits) rounded to the nearest e4m3 value, ties to even: steps of 2^(e - 3) in the binade 2^e, e >= -6."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact_weight(w, cols):
    if w.dim() == 1:
        return w.double()
    return torch.cat([w[l].double().repeat(2 * l + 1) for l in range(4)])


def exact_norm(st):
    case = st["case"]
    s = st["x"].double() if st["residual"] is None else st["x"].double() + st["residual"].double()
    size = (torch.einsum("ij,ij->i", s, s) / case["cols"] + EPS).sqrt()
    y = s / size[:, None] * exact_weight(st["w"], case["cols"])
    if not case["quantize"]:
        return y, s
    top = y.abs().max(1).values
    scale = top / E4M3_MAX
    scale[top < TINY] = 1.0
    return e4m3_values(y / scale[:, None]), scale, s


def exact_norm_grad(st):
    case = st["case"]
    s, g = st["s"].double(), st["g"].double()
    cols = case["cols"]
    var = torch.einsum("ij,ij->i", s, s) / cols + EPS
    h = g * exact_weight(st["w"], cols)
    g_x = h / var.sqrt()[:, None] - s * (torch.einsum("ij,ij->i", h, s) / (cols * var * var.sqrt()))[:, None]
    if st["g_s"] is not None:
        g_x += st["g_s"].double()
    g_w = torch.einsum("ij,ij,i->j", g, s, 1.0 / var.sqrt())
    if case["degrees"]:
        g_w = torch.stack([p.sum(0) for p in torch.split(g_w.view(16, cols // 16), [1, 3, 5, 7])])
    return g_x, g_w


def normal_cdf(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def exact_act(z, act):
    return z / (1.0 + torch.exp(-z)) if act == "silu" else z * normal_cdf(z) if act == "gelu" else z


def exact_slope(z, act):
    if act == "silu":
        return (1.0 + torch.exp(-z) + z * torch.exp(-z)) / (1.0 + torch.exp(-z)) ** 2
    return normal_cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def exact_dense(st):
    case = st["case"]
    x, w = st["x"].double(), st["w"].double()
    if st["x_scale"] is not None:
        x, w = x * st["x_scale"].double()[:, None], w * st["w_scale"].double()[:, None]
    z = torch.einsum("mk,nk->mn", x, w)
    if st["b"] is not None:
        z += st["b"].double()
    y = exact_act(z, case["act"])
    if st["residual"] is not None:
        y = y + st["residual"].double()
    return (y, z) if case["keep_z"] else y


def exact_dense_grad(st):
    g = st["g"].double()
    if st["z"] is not None:
        g = g * exact_slope(st["z"].double(), st["case"]["act"])
    return (torch.einsum("mn,nk->mk", g, st["w"].double()), torch.einsum("mn,mk->nk", g, st["x"].double()),
            torch.einsum("mn->n", g))


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": exact_norm, "norm_grad": exact_norm_grad, "dense": exact_dense,
            "dense_grad": exact_dense_grad}[case["op"]](st)
