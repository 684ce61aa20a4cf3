"""Layer norm over sharded volumes against the fp64 definition.

Tolerances, element by element: a bf16 output is rounded once (2^-8 of its
value); everything before is fp32 sums of C terms and a handful of products,
taken as 2^-24 * (8 + 2 sqrt(C)) of the absolute values that enter:
  y       |xhat gamma| + |beta| + |gamma| (1 + |mean| rstd)
  dx      rstd (|g| + mean|g| + |xhat| mean|g xhat|), times (1 + |mean| rstd) for
          what the error of xhat brings
  dgamma  sums over the cells of |dy| (|xhat| + |mean| rstd + 1); dbeta of |dy|
"""
import math

import numpy as np
import pytest
import torch

import synth
from helpers import say
from oracle import tokens

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


class Shards:
    """Shard buffers of a channels-last volume, margins filled with `margin`."""

    def __init__(self, lib, spatial, sizes, batch, channels, halo, dtype, margin=math.nan):
        nd = len(spatial)
        self.plan = lib.st_plan_shards(nd, batch, channels, spatial, sizes, [halo] * nd, dtype)
        self.halo = halo
        self.infos = [self.plan.shard_info(i) for i in range(self.plan.num_shards)]
        self.bufs = [torch.full(self.plan.padded_shape(i), margin, dtype=TORCH[dtype], device="cuda")
                     for i in range(self.plan.num_shards)]

    def interior(self, i):
        h = self.halo
        return self.bufs[i][(slice(None), *[slice(h, h + e) for e in self.infos[i]["extent"]])]

    def where(self, i):
        inf = self.infos[i]
        return (slice(None), *[slice(o, o + e) for o, e in zip(inf["offset"], inf["extent"])])

    def load(self, x):
        for i in range(len(self.bufs)):
            self.interior(i).copy_(x[self.where(i)])
        return self

    def gather(self, like):
        out = torch.empty(like.shape, dtype=self.bufs[0].dtype)
        for i in range(len(self.bufs)):
            out[self.where(i)] = self.interior(i).cpu()
        return out

    def cells(self, i):
        return self.interior(i).numel() // self.plan.channels


def make(spatial, batch, c, xt, yt, seed=0, offset=0.5):
    rng = np.random.default_rng(seed)
    shape = (batch, *spatial, c)
    x = torch.from_numpy(rng.normal(size=shape) * rng.uniform(0.2, 2, size=c) + offset).to(TORCH[xt])
    dy = torch.from_numpy(rng.normal(size=shape)).to(TORCH[yt])
    gamma = torch.from_numpy(rng.normal(size=c) * 0.3 + 1).float()
    beta = torch.from_numpy(rng.normal(size=c) * 0.3).float()
    return x, dy, gamma, beta


def run(lib, x, dy, gamma, beta, spatial, sizes, xt, yt, dxt, halos, eps=1e-5, affine=True):
    batch, c = x.shape[0], x.shape[-1]
    xs = Shards(lib, spatial, sizes, batch, c, halos[0], xt).load(x)
    ys = Shards(lib, spatial, sizes, batch, c, halos[1], yt, margin=5.0)
    dys = Shards(lib, spatial, sizes, batch, c, halos[1], yt).load(dy)
    dxs = Shards(lib, spatial, sizes, batch, c, halos[2], dxt, margin=5.0)
    g, b = (gamma.cuda(), beta.cuda()) if affine else (None, None)
    n = sum(xs.cells(i) for i in range(len(xs.bufs)))
    stats = torch.full((n + 1, 2), 9.0, device="cuda")
    lib.st_layernorm_sharded(xs.plan, xs.bufs, g, b, eps, ys.plan, ys.bufs, stats)
    need = lib.st_layernorm_backward_workspace_bytes(xs.plan)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    dg, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    lib.st_layernorm_backward(xs.plan, xs.bufs, dys.plan, dys.bufs, g, stats, dxs.plan, dxs.bufs, dg, db, ws[:need])
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0x5A).all()) and bool((stats[n:] == 9.0).all())
    for s in (ys, dxs):                                   # margins are not written
        for i, buf in enumerate(s.bufs):
            left = buf.clone()
            Shards.interior(s, i).numel()
            h = s.halo
            left[(slice(None), *[slice(h, h + e) for e in s.infos[i]["extent"]])] = 5.0
            assert bool((left == 5.0).all())
    return {"y": ys.gather(x), "dx": dxs.gather(x), "dgamma": dg.cpu(), "dbeta": db.cpu(), "stats": stats[:n].cpu(), "xs": xs}


def check(r, x, dy, gamma, beta, yt, dxt, eps=1e-5, affine=True):
    x64, dy64 = x.double().numpy(), dy.double().numpy()
    g64, b64 = (gamma.double().numpy(), beta.double().numpy()) if affine else (np.ones(x.shape[-1]), np.zeros(x.shape[-1]))
    y, mean, rstd = tokens.layer_norm(x64, g64, b64, eps)
    dx, dg, db = tokens.layer_norm_backward(x64, dy64, g64, eps)
    c = x.shape[-1]
    u = 2.0 ** -24 * (8 + 2 * math.sqrt(c))
    lean = (1 + np.abs(mean) * rstd)[..., None]
    xhat = (x64 - mean[..., None]) * rstd[..., None]
    g = np.abs(dy64 * g64)
    by = np.abs(xhat * g64) + np.abs(b64) + np.abs(g64) * lean
    bdx = rstd[..., None] * (g + g.mean(-1, keepdims=True) + np.abs(xhat) * (g * np.abs(xhat)).mean(-1, keepdims=True)) * lean
    cells = x64.size // c
    axes = tuple(range(x64.ndim - 1))
    us = 2.0 ** -24 * (16 + 2 * math.sqrt(cells))          # and the sums over the cells
    for name, want, bound, t, e in (("y", y, by, yt, u), ("dx", dx, bdx, dxt, u),
                                    ("dgamma", dg, (np.abs(dy64) * (np.abs(xhat) + lean)).sum(axes), "f32", us),
                                    ("dbeta", db, np.abs(dy64).sum(axes), "f32", us)):
        tol = e * bound + (2.0 ** -8 * np.abs(want) * 1.001 if t == "bf16" else 0)
        off = np.abs(r[name].double().numpy() - want)
        assert np.all(off <= tol), f"{name}: off {off.max()}, over by {np.max(off - tol)}"
    got = np.zeros((2, *mean.shape))
    at = 0
    for i in range(len(r["xs"].bufs)):
        n = r["xs"].cells(i)
        w = r["xs"].where(i)
        got[(0, *w)], got[(1, *w)] = (r["stats"][at:at + n, j].double().numpy().reshape(mean[w].shape) for j in (0, 1))
        at += n
    assert np.all(np.abs(got[0] - mean) <= u * np.abs(x64).mean(-1) + 1e-30)
    assert np.all(np.abs(got[1] - rstd) <= u * rstd * lean[..., 0])


@pytest.mark.parametrize("xt,yt,dxt", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"), ("bf16", "f32", "f32")])
@pytest.mark.parametrize("c", [8, 16, 64, 256, 20, 33, 7, 1000])
def test_widths(gpu_lib, c, xt, yt, dxt):
    say(f"layer norm C={c} {xt}->{yt} dx {dxt}")
    spatial, sizes = (7, 19), ((3, 4), (12, 7))
    x, dy, gamma, beta = make(spatial, 2, c, xt, yt)
    r = run(gpu_lib, x, dy, gamma, beta, spatial, sizes, xt, yt, dxt, (0, 1, 2))
    check(r, x, dy, gamma, beta, yt, dxt)


@pytest.mark.parametrize("c", [1025, 2056, 4100, 4104, 8200, 16384, 16383, 520, 1032, 2064])
def test_wide_cells(gpu_lib, c):
    """Cells held by a whole workgroup, each kernel variant."""
    for xt in ("f32", "bf16"):
        say(f"layer norm C={c} {xt}")
        x, dy, gamma, beta = make((1, 5), 1, c, xt, xt)
        r = run(gpu_lib, x, dy, gamma, beta, (1, 5), ((1,), (5,)), xt, xt, xt, (0, 0, 0))
        check(r, x, dy, gamma, beta, xt, xt)


def test_volume_and_shards(gpu_lib):
    """A 3D volume: a cell's bits do not depend on the shard plan, and the sums
    over cells agree to fp32."""
    spatial = (6, 7, 9)
    x, dy, gamma, beta = make(spatial, 1, 32, "f32", "bf16", offset=3.0)
    a = run(gpu_lib, x, dy, gamma, beta, spatial, ((6,), (7,), (9,)), "f32", "bf16", "f32", (0, 0, 0))
    b = run(gpu_lib, x, dy, gamma, beta, spatial, ((1, 5), (4, 3), (2, 7)), "f32", "bf16", "f32", (1, 1, 0))
    check(a, x, dy, gamma, beta, "bf16", "f32")
    check(b, x, dy, gamma, beta, "bf16", "f32")
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["dx"], b["dx"])


def test_repository_volume(gpu_lib):
    """The 32^3 volume of the fp32 workload, split 17/15, its 8 output channels."""
    wl = synth.workload("vol32_c4to8_k3_fp32")
    x, dy, gamma, beta = make(wl.spatial, 1, wl.cout, "f32", "f32")
    r = run(gpu_lib, x, dy, gamma, beta, wl.spatial, wl.shards, "f32", "f32", "f32", (0, 0, 1))
    check(r, x, dy, gamma, beta, "f32", "f32")


def test_no_affine_and_eps(gpu_lib):
    x, dy, gamma, beta = make((4, 5), 1, 48, "f32", "f32")
    x[0, 1, 2] = 2.5                                      # a constant cell: variance 0
    r = run(gpu_lib, x, dy, gamma, beta, (4, 5), ((4,), (5,)), "f32", "f32", "f32", (0, 0, 0), eps=1e-3, affine=False)
    check(r, x, dy, gamma, beta, "f32", "f32", eps=1e-3, affine=False)
    assert bool((r["y"][0, 1, 2] == 0).all())


def test_special_values_stay_in_their_cell(gpu_lib):
    x, dy, gamma, beta = make((4, 5), 1, 48, "bf16", "bf16")
    clean = run(gpu_lib, x, dy, gamma, beta, (4, 5), ((4,), (5,)), "bf16", "bf16", "bf16", (0, 0, 0))
    bad = x.clone()
    bad[0, 2, 3, 7] = math.inf
    r = run(gpu_lib, bad, dy, gamma, beta, (4, 5), ((4,), (5,)), "bf16", "bf16", "bf16", (0, 0, 0))
    assert bool(torch.isnan(r["y"][0, 2, 3].float()).any())
    for n in ("y", "dx"):
        r[n][0, 2, 3] = clean[n][0, 2, 3]
        assert torch.equal(r[n], clean[n]), n


def test_in_place_and_optional_outputs(gpu_lib):
    x, dy, gamma, beta = make((4, 9), 1, 64, "bf16", "bf16")
    want = run(gpu_lib, x, dy, gamma, beta, (4, 9), ((4,), (9,)), "bf16", "bf16", "bf16", (0, 0, 0))
    s = Shards(gpu_lib, (4, 9), ((4,), (9,)), 1, 64, 0, "bf16").load(x)
    gpu_lib.st_layernorm_sharded(s.plan, s.bufs, gamma.cuda(), beta.cuda(), 1e-5, s.plan, s.bufs)
    assert torch.equal(s.gather(x), want["y"])
    xs = Shards(gpu_lib, (4, 9), ((4,), (9,)), 1, 64, 0, "bf16").load(x)
    s.load(dy)
    ws = torch.empty(gpu_lib.st_layernorm_backward_workspace_bytes(s.plan), dtype=torch.uint8, device="cuda")
    db = torch.empty(64, device="cuda")
    gpu_lib.st_layernorm_backward(xs.plan, xs.bufs, s.plan, s.bufs, gamma.cuda(), want["stats"].cuda(), s.plan, s.bufs, None, db, ws)
    assert torch.equal(s.gather(x), want["dx"]) and torch.equal(db.cpu(), want["dbeta"])


def test_gradient_against_differences(gpu_lib):
    """fp32: directional derivative of sum(y * dy) by central differences of the
    library's forward pass, h = 2^-6: truncation ~ h^2 and rounding
    ~ 2^-22 |f| / h stay below 1% of the gradient's norm."""
    spatial, sizes = (3, 11), ((3,), (11,))
    x, dy, gamma, beta = make(spatial, 1, 40, "f32", "f32")
    r = run(gpu_lib, x, dy, gamma, beta, spatial, sizes, "f32", "f32", "f32", (0, 0, 0))
    rng = np.random.default_rng(9)
    h = 2.0 ** -6
    for name, at in (("dx", 0), ("dgamma", 1), ("dbeta", 2)):
        args = [x, gamma, beta]
        t = torch.from_numpy(rng.normal(size=tuple(args[at].shape)))
        f = []
        for sign in (1, -1):
            m = list(args)
            m[at] = (args[at].double() + sign * h * t).float()
            y = run(gpu_lib, m[0], dy, m[1], m[2], spatial, sizes, "f32", "f32", "f32", (0, 0, 0))["y"]
            f.append(float((y.double() * dy.double()).sum()))
        got, want = (f[0] - f[1]) / (2 * h), float((r[name].double() * t).sum())
        assert abs(got - want) <= 0.02 * float(torch.linalg.vector_norm(r[name].double())), name


def test_offsets_past_32_bits(gpu_lib):
    """A shard of 2.2e9 values: its last cells are those of a small shard."""
    n, c = 270000, 8200
    x = torch.empty(n, c, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    g = torch.randn(c, device="cuda")

    def both(rows):
        m = len(rows)
        plan = gpu_lib.st_plan_shards(2, 1, c, (1, m), ((1,), (m,)), (0, 0), "bf16")
        y, dx, stats = torch.empty_like(rows), torch.empty_like(rows), torch.empty(m, 2, device="cuda")
        gpu_lib.st_layernorm_sharded(plan, [rows], g, None, 1e-5, plan, [y], stats)
        ws = torch.empty(gpu_lib.st_layernorm_backward_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
        gpu_lib.st_layernorm_backward(plan, [rows], plan, [y], g, stats, plan, [dx], None, None, ws)
        return y[-40:].clone(), dx[-40:].clone(), stats[-40:].clone()

    assert all(torch.equal(a, b) for a, b in zip(both(x), both(x[-40:].clone())))


def test_refusals_on_the_gpu(gpu_lib):
    s = Shards(gpu_lib, (4, 9), ((4,), (9,)), 1, 64, 0, "f32", margin=0.0)
    o = Shards(gpu_lib, (4, 9), ((3, 1), (9,)), 1, 64, 0, "f32", margin=0.0)
    d = Shards(gpu_lib, (4, 9), ((4,), (9,)), 1, 32, 0, "f32", margin=0.0)

    def status(f):
        with pytest.raises(gpu_lib.ShardConvError) as e:
            f()
        return e.value.status

    ln = gpu_lib.st_layernorm_sharded
    assert status(lambda: ln(s.plan, s.bufs, None, None, 1e-5, o.plan, o.bufs)) == 2
    assert status(lambda: ln(s.plan, s.bufs, None, None, 1e-5, d.plan, d.bufs)) == 2
    assert status(lambda: ln(s.plan, s.bufs, None, None, -1.0, s.plan, s.bufs)) == 1
    assert status(lambda: ln(s.plan, s.bufs, None, None, math.nan, s.plan, s.bufs)) == 1
    wide = gpu_lib.st_plan_shards(2, 1, 16392, (1, 1), ((1,), (1,)), (0, 0), "f32")
    big = [torch.zeros(16392, device="cuda")]
    assert status(lambda: ln(wide, big, None, None, 1e-5, wide, big)) == 4
    stats = torch.zeros(36, 2, device="cuda")
    assert status(lambda: gpu_lib.st_layernorm_backward(s.plan, s.bufs, s.plan, s.bufs, None, stats, s.plan, s.bufs, None, None, None)) == 5
    g = torch.zeros(65, device="cuda")[1:]
    assert status(lambda: ln(s.plan, s.bufs, g, None, 1e-5, s.plan, s.bufs)) == 7


def test_more_cells_than_one_launch_holds(gpu_lib):
    """2^28 cells of 33 channels are 2^24 workgroups of 256 threads, one more than
    a launch takes: the cells around the cut and the last ones are those of a
    small call.  The backward pass has a fixed number of workgroups."""
    n, c = (1 << 28) + 37, 33
    x = torch.empty(n, c, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    g = torch.randn(c, device="cuda")
    ends = [slice(0, 20), slice((1 << 28) - 40, (1 << 28) + 17), slice(n - 21, n)]

    def forward(rows):
        plan = gpu_lib.st_plan_shards(2, 1, c, (1, len(rows)), ((1,), (len(rows),)), (0, 0), "bf16")
        gpu_lib.st_layernorm_sharded(plan, [rows], g, None, 1e-5, plan, [rows])
        return rows

    want = [forward(x[e].clone()) for e in ends]
    forward(x)
    assert all(torch.equal(x[e], w) for e, w in zip(ends, want))
