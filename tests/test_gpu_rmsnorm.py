"""RMS norm with the residual's addition against the fp64 definition.

Tolerances, element by element: sums of C terms and a handful of products in
fp32, 2^-24 (8 + 2 sqrt(C)) of the magnitudes that enter, and one rounding to
the output's type.  The sum is exact: one fp32 addition, one rounding to its type.
"""
import math

import numpy as np
import pytest
import torch

from helpers import say
from mlp_helpers import Operand, TORCH, npy, rounding, sums, within
from oracle import mlp

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 7), (1, 2048), (9, 32), (70, 64), (33, 100), (5, 1000), (6, 1001), (4, 4096), (3, 4100), (2, 8200), (2, 16384), (3, 16383), (4099, 40)]


def make(rows, c, x, res, seed=0):
    rng = np.random.default_rng(seed)
    a = torch.from_numpy(rng.normal(size=(rows, c)) * rng.uniform(0.1, 2, size=c)).to(TORCH[x])
    b = torch.from_numpy(rng.normal(size=(rows, c))).to(TORCH[res]) if res else None
    gamma = torch.from_numpy(1 + 0.3 * rng.normal(size=c)).float()
    dy = rng.normal(size=(2, rows, c))
    return a, b, gamma, torch.from_numpy(dy[0]), torch.from_numpy(dy[1])


@pytest.mark.parametrize("rows,c", SHAPES)
@pytest.mark.parametrize("x,res,total,y", [("f32", "bf16", "f32", "bf16"), ("bf16", "bf16", "bf16", "bf16"),
                                           ("f32", "", "", "f32"), ("bf16", "f32", "bf16", "f32")])
@pytest.mark.parametrize("extra", [0, 24])
def test_forward_and_backward(gpu_lib, rows, c, x, res, total, y, extra):
    say(f"rms norm {rows}x{c} {x}+{res}->{total},{y} extra {extra}")
    eps = 1e-6
    a, b, gamma, dyv, dtv = make(rows, c, x, res, rows + c)
    ax = Operand(gpu_lib, rows, c, x, a, extra)
    bx = Operand(gpu_lib, rows, c, res, b, extra) if res else None
    tx = Operand(gpu_lib, rows, c, total, extra=extra) if total else None
    yx, y8 = Operand(gpu_lib, rows, c, y, extra=extra), Operand(gpu_lib, rows, c, "mx8", extra=extra)
    g, rstd = gamma.cuda(), torch.full((rows + 4,), 7.0, device="cuda")
    gpu_lib.st_rmsnorm(ax.t, bx.t if bx else None, g, eps, total=tx.t if tx else None, y=yx.t, y8=y8.t, rstd=rstd)
    torch.cuda.synchronize()
    s = a.float() + b.float() if res else a.float()
    s = s.to(TORCH[total]) if total else s
    s64, g64 = npy(s), npy(gamma)
    if tx:
        tx.check_guards()
        assert np.array_equal(tx.values(), s64)
    want, r = mlp.rms_norm(s64, g64, eps)
    u = sums(c)
    yx.check_guards()
    y8.check_guards()
    within("rstd", npy(rstd[:rows]), r, u * r)
    assert bool((rstd[rows:] == 7.0).all())
    within("y", yx.values(), want, u * np.abs(want) + rounding(want, y))
    within("y8", y8.values(), want, u * np.abs(want) + rounding(want, "mx8"))

    for kept in {total or "f32", "mx8"}:
        sk = Operand(gpu_lib, rows, c, kept, s, extra)
        for dtot, dxt in (("f32", "bf16"), ("", "f32"), ("bf16", "bf16")):
            dyx = Operand(gpu_lib, rows, c, y, dyv, extra)
            dtx = Operand(gpu_lib, rows, c, dtot, dtv, extra) if dtot else None
            dx = Operand(gpu_lib, rows, c, dxt, extra=extra)
            dg = torch.full((c + 4,), 7.0, device="cuda")
            need = gpu_lib.st_rmsnorm_backward_workspace_bytes(rows, c)
            ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
            gpu_lib.st_rmsnorm_backward(sk.t, dyx.t, dtx.t if dtx else None, g, rstd[:rows], dx.t, dg[:c], ws[:need])
            torch.cuda.synchronize()
            dx.check_guards()
            assert bool((ws[need:] == 0x5A).all()) and bool((dg[c:] == 7.0).all())
            wdx, wdg = mlp.rms_norm_backward(sk.values(), dyx.values(), dtx.values() if dtx else None, g64, r)
            xh, h = np.abs(sk.values()) * r[:, None], np.abs(dyx.values() * g64)
            mag = r[:, None] * (h + xh * (h * xh).mean(-1, keepdims=True)) + (np.abs(dtx.values()) if dtx else 0)
            within(f"dx {kept} {dtot} {dxt}", dx.values(), wdx, 2 * u * mag + rounding(wdx, dxt))
            within("dgamma", npy(dg[:c]), wdg, (u + sums(rows)) * (np.abs(dyx.values()) * xh).sum(0))


def test_in_place(gpu_lib):
    """The stream's own buffer takes the sum; dx takes dtotal's or dy's."""
    rows, c = 50, 256
    a, b, gamma, dyv, dtv = make(rows, c, "f32", "bf16")
    apart = {n: Operand(gpu_lib, rows, c, "f32", a) for n in "xs"}
    bx, y = Operand(gpu_lib, rows, c, "bf16", b), [Operand(gpu_lib, rows, c, "bf16") for _ in range(2)]
    g, rstd = gamma.cuda(), torch.empty(rows, device="cuda")
    gpu_lib.st_rmsnorm(apart["x"].t, bx.t, g, 1e-6, total=apart["s"].t, y=y[0].t, rstd=rstd)
    gpu_lib.st_rmsnorm(apart["x"].t, bx.t, g, 1e-6, total=apart["x"].t, y=y[1].t, rstd=rstd)
    assert torch.equal(apart["x"].t, apart["s"].t) and torch.equal(y[0].t, y[1].t)
    ws = torch.empty(gpu_lib.st_rmsnorm_backward_workspace_bytes(rows, c), dtype=torch.uint8, device="cuda")
    dy, dt, dx = (Operand(gpu_lib, rows, c, "f32", v) for v in (dyv, dtv, dtv))
    want = Operand(gpu_lib, rows, c, "f32")
    dg = [torch.empty(c, device="cuda") for _ in range(3)]
    args = (apart["s"].t, dy.t, dt.t, g, rstd)
    gpu_lib.st_rmsnorm_backward(*args, want.t, dg[0], ws)
    gpu_lib.st_rmsnorm_backward(apart["s"].t, dy.t, dx.t, g, rstd, dx.t, dg[1], ws)
    assert torch.equal(dx.t, want.t) and torch.equal(dg[0], dg[1])
    gpu_lib.st_rmsnorm_backward(*args, dy.t, dg[2], ws)
    assert torch.equal(dy.t, want.t) and torch.equal(dg[0], dg[2])


def test_empty_zero_and_special_rows(gpu_lib):
    """No rows: nothing but a cleared dgamma.  A row of zeros: y = 0, rstd = eps^-1/2.
    A NaN stays in its own row."""
    c = 64
    none = torch.empty(0, c, device="cuda")
    gpu_lib.st_rmsnorm(none, None, None, 1e-6, y=none.clone())
    dg = torch.ones(c, device="cuda")
    ws = torch.empty(gpu_lib.st_rmsnorm_backward_workspace_bytes(0, c), dtype=torch.uint8, device="cuda")
    gpu_lib.st_rmsnorm_backward(none, none, None, None, torch.empty(0, device="cuda"), none.clone(), dg, ws)
    assert bool((dg == 0).all())
    x = torch.ones(3, c, device="cuda")
    x[0] = 0
    x[2, 5] = math.nan
    y, r = torch.empty_like(x), torch.empty(3, device="cuda")
    y8 = gpu_lib.mx8_empty(3, c)
    gpu_lib.st_rmsnorm(x, None, None, 1e-6, y=y, y8=y8, rstd=r)
    assert bool((y[0] == 0).all()) and abs(float(r[0]) - 1e3) < 1e-3 and bool(torch.isnan(y[2]).all())
    assert abs(float(y[1].mean()) - 1) < 1e-5
    back = torch.empty_like(x)
    gpu_lib.st_mx8_load(y8, back)
    assert bool(torch.isnan(back[2]).all()) and bool((back[0] == 0).all()) and bool((back[1] == 1).all())


def test_same_bits_twice_and_without_outputs(gpu_lib):
    rows, c = 3000, 520
    a, b, gamma, dyv, dtv = make(rows, c, "bf16", "bf16")
    ops = [Operand(gpu_lib, rows, c, "bf16", v) for v in (a, dyv, dtv)]
    g, rstd = gamma.cuda(), torch.empty(rows, device="cuda")
    gpu_lib.st_rmsnorm(ops[0].t, None, g, 1e-6, rstd=rstd)
    ws = torch.empty(gpu_lib.st_rmsnorm_backward_workspace_bytes(rows, c), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(2):
        dx, dg = torch.empty(rows, c, device="cuda"), torch.empty(c, device="cuda")
        gpu_lib.st_rmsnorm_backward(ops[0].t, ops[1].t, ops[2].t, g, rstd, dx, dg, ws)
        got.append((dx, dg))
    dx = torch.empty(rows, c, device="cuda")
    gpu_lib.st_rmsnorm_backward(ops[0].t, ops[1].t, ops[2].t, g, rstd, dx, None, None)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and torch.equal(dx, got[0][0])
