"""Small, self-contained invocations of single kernel families, for profilers.

    python -m edge_message_passing_b200.kernel_cases <case> [--iters K]

Cases (seeded synthetic inputs, sizes chosen so that buffers exceed the 126 MB L2
while the device footprint stays at a few GB):
  so2      one 8192-row cohort of the SO(2) mixing (C = 128), forward map
  so2t     the same, transpose (adjoint) map
  step512  one energy + force step of the N=512 diamond model (C = 128, 3 layers)
  step4096 one energy + force step of the N=4096 diamond model (the benchmark workload;
           for one-pass launch lists only: its workspace is several GB)
  chain    the folded radial chain at E = 647170, forward + input gradient
  norm     RMS norm of 16384 x 2048 bf16 rows with a residual, to e4m3, weights per degree
  normg    its gradient on 16384 x 2048 FP32 rows
  normodd  RMS norm of 80896 x 515 bf16 rows (off 16-byte boundaries)
  dense64  dense layer 161792 x 64 -> 512 with SiLU, FP32 (k of one chunk)
  dense512 dense layer 40448 x 512 -> 512, FP32
  dense16  dense layer 16384 x 2048 -> 2048, bf16
  dense8   dense layer 65536 x 2048 -> 512 of e4m3 with scales, SiLU and a residual
  denseg   gradient of a dense layer 40448 x 128 -> 512 with SiLU, FP32
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


ROW_CASES = ("norm", "normg", "normodd", "dense64", "dense512", "dense16", "dense8", "denseg")


def row_case(name: str):
    """One call of a row-wise operator, as a function without arguments."""
    import torch

    import edge_message_passing_b200 as emp

    def t(*shape, dtype=torch.float32):
        return torch.randn(shape, device="cuda").to(dtype)

    bf16, e4m3 = torch.bfloat16, torch.float8_e4m3fn
    if name == "norm":
        x, r, w = t(16384, 2048, dtype=bf16), t(16384, 2048, dtype=bf16), t(4, 128, dtype=bf16)
        return lambda: emp.mp_rms_norm(x, w, residual=r, quantize=True)
    if name == "normg":
        g, s, w, gs = t(16384, 2048), t(16384, 2048), t(4, 128), t(16384, 2048)
        return lambda: emp.mp_rms_norm_grad(g, s, w, g_s=gs)
    if name == "normodd":
        x, w = t(80896, 515, dtype=bf16), t(515, dtype=bf16)
        return lambda: emp.mp_rms_norm(x, w)
    if name == "dense8":
        x, w, r = t(65536, 2048).to(e4m3), t(512, 2048).to(e4m3), t(65536, 512, dtype=bf16)
        xs, ws = torch.rand(65536, device="cuda"), torch.rand(512, device="cuda")
        return lambda: emp.mp_dense(x, w, activation="silu", residual=r, x_scale=xs, w_scale=ws)
    rows, K, N, dtype, act = {"dense64": (161792, 64, 512, torch.float32, "silu"), "dense512": (40448, 512, 512, torch.float32, "none"),
                              "dense16": (16384, 2048, 2048, bf16, "none"),
                              "denseg": (40448, 128, 512, torch.float32, "silu")}[name]
    x, w, b = t(rows, K, dtype=dtype), t(N, K, dtype=dtype), t(N, dtype=dtype)
    if name != "denseg":
        return lambda: emp.mp_dense(x, w, b, activation=act)
    g, z = t(rows, N, dtype=dtype), t(rows, N, dtype=dtype)
    return lambda: emp.mp_dense_grad(g, x, w, z=z, activation=act)


def main() -> int:
    import torch

    import edge_message_passing_b200 as emp
    import synth

    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=["so2", "so2t", "step512", "step4096", "chain", *ROW_CASES])
    ap.add_argument("--iters", type=int, default=3)
    a = ap.parse_args()
    torch.cuda.set_device(0)
    if a.case in ("so2", "so2t"):
        spec = synth.ModelSpec(C=128, n_layers=1)
        model = emp.Model(spec, synth.draw_weights(spec, np.random.default_rng(0)))
        X = torch.randn((8192, 16 * 128), device="cuda")
        for _ in range(a.iters):
            emp.mp_so2_mix(model, 0, X, transpose=a.case == "so2t")
    elif a.case in ("step512", "step4096"):
        w = synth.workload("n512_diamond" if a.case == "step512" else "n4096_diamond")
        model = emp.Model(w.spec, w.weights)
        g = emp.nl_build(torch.from_numpy(w.structure.pos).cuda(), w.structure.box, w.spec.cutoff)
        sp = torch.from_numpy(w.structure.species).cuda()
        for _ in range(a.iters):
            emp.mp_energy_forces(model, g, sp)
    elif a.case in ROW_CASES:
        call = row_case(a.case)
        for _ in range(a.iters):
            call()
    else:
        ci = synth.chain_inputs()
        ch = emp.Chain(ci.U, ci.M)
        x, gk, gy = (torch.from_numpy(t).cuda() for t in (ci.x, ci.g_kc, ci.g_y0))
        for _ in range(a.iters):
            emp.mp_radial_chain(ch, x, gk, gy)
    torch.cuda.synchronize()
    err = emp.last_device_error()
    print(f"{a.case}: done, device error word {err}")
    return 0 if err == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
