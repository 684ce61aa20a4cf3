"""Matrix products with bias, activation and residual, and their gradients,
against the fp64 definition.

Tolerances, element by element: a sum of K products in fp32 is off by 2^-24 (8 +
2 sqrt(K)) of the sum of magnitudes; the activations' slopes stay below 1.13 and
their own steps cost a few 2^-24 (exponents of up to z^2); every rounding to
bf16 costs 2^-8 and to e4m3 2^-4 of the value.  The 8-bit instructions (outputs
that are no fp32) cut each of eight products 13 bits below the largest one's
leading bit: at most seven lose bits, each less than 2^-13 of the largest.  With bf16 products the backward
pass rounds p = dy * act'(pre) to bf16: 2^-8 of every term.
"""
import math

import numpy as np
import pytest
import torch

from helpers import say
from mlp_helpers import Operand, TORCH, npy, rounding, sums, within
from oracle import mlp

pytestmark = pytest.mark.gpu


def make(lib, m, k, n, dtype, seed=0, extra=0):
    rng = np.random.default_rng(seed)
    x = Operand(lib, m, k, dtype, torch.from_numpy(rng.normal(size=(m, k)) * rng.uniform(0.2, 2, size=k)), extra)
    w = Operand(lib, n, k, dtype, torch.from_numpy(rng.normal(size=(n, k)) / math.sqrt(k)), extra)
    return rng, x, w


def act_error(z, act):
    """Of the activation's fp32 steps (its arguments' error apart)."""
    return 0 if act in ("none", "relu") else 2.0 ** -24 * (16 + 2 * z * z) * np.minimum(np.abs(z), 1) * np.exp(-np.minimum(z * z, 80) / 4) + 2.0 ** -22 * np.abs(z)


def cut8(x, w):
    """Sum over the groups of eight steps of the largest product."""
    total = np.zeros((x.shape[0], w.shape[0]))
    for lo in range(0, x.shape[1], 8):
        top = np.zeros_like(total)
        for k in range(lo, min(lo + 8, x.shape[1])):
            np.maximum(top, np.abs(x[:, k, None] * w[None, :, k]), out=top)
        total += top
    return total


def forward(lib, m, k, n, dtype, act, res, y, pre, bias=True, extra=0, seed=0):
    rng, x, w = make(lib, m, k, n, dtype, seed, extra)
    b = torch.from_numpy(0.3 * rng.normal(size=n)).float() if bias else None
    r = Operand(lib, m, n, res, torch.from_numpy(rng.normal(size=(m, n))), extra) if res else None
    yo, po = Operand(lib, m, n, y, extra=extra), Operand(lib, m, n, pre, extra=extra) if pre else None
    need = lib.st_linear_workspace_bytes(m, k, n, dtype)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    lib.st_linear(x.t, w.t, b.cuda() if bias else None, yo.t, act=act, residual=r.t if r else None, pre=po.t if po else None,
                  workspace=ws[:need])
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0x5A).all())
    yo.check_guards()
    xv, wv = x.values(), w.values()
    want, z = mlp.linear(xv, wv, npy(b) if bias else None, act, r.values() if r else None)
    dz = sums(k) * (np.abs(xv) @ np.abs(wv).T + (np.abs(npy(b)) if bias else 0))
    if dtype == "mx8" and "f32" not in (y, pre):
        dz = dz + 7 * 2.0 ** -13 * cut8(xv, wv)
    dy = 1.13 * dz + act_error(z, act) + 2.0 ** -24 * (np.abs(want) + (np.abs(r.values()) if r else 0))
    within("y", yo.values(), want, dy + rounding(np.abs(want) + dy, y))
    if po:
        po.check_guards()
        within("pre", po.values(), z, dz + rounding(np.abs(z) + dz, pre))


# one token, few, odd, a tile, past a tile; contractions below, at and past a stage
SIZES = [(1, 8, 8), (1, 64, 256), (1, 2048, 520), (3, 40, 7), (17, 33, 65), (33, 1000, 257), (64, 512, 128), (65, 96, 100),
         (130, 64, 300), (200, 4104, 40), (257, 1001, 131), (700, 256, 516), (1, 1, 1), (5, 7, 3)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32", "mx8"])
@pytest.mark.parametrize("extra", [0, 40])
def test_products(gpu_lib, m, k, n, dtype, extra):
    say(f"linear {m}x{k}x{n} {dtype} extra {extra}")
    y = "f32" if (m + n) % 2 else "bf16"
    forward(gpu_lib, m, k, n, dtype, "none", "", y, "", extra=extra, seed=m + k + n)
    forward(gpu_lib, m, k, n, dtype, "none", "", y, "", bias=False, extra=extra, seed=m + k)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("res", ["", "f32", "bf16"])
@pytest.mark.parametrize("y,pre", [("bf16", ""), ("f32", "f32"), ("mx8", "bf16"), ("bf16", "mx8")])
@pytest.mark.parametrize("m,k,n", [(2, 64, 100), (150, 128, 200)])
def test_epilogues(gpu_lib, act, res, y, pre, m, k, n):
    say(f"linear {m}x{k}x{n} {act} {res} {y} {pre}")
    for dtype in ("bf16", "f32", "mx8"):
        forward(gpu_lib, m, k, n, dtype, act, res, y, pre, seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mx8"])
@pytest.mark.parametrize("m,k,n", [(512, 256, 768), (300, 9000, 260), (1500, 96, 1100), (4, 8192, 96)])
def test_many_tiles_and_splits(gpu_lib, dtype, m, k, n):
    say(f"linear {m}x{k}x{n} {dtype}")
    forward(gpu_lib, m, k, n, dtype, "gelu", "bf16", "f32", "bf16", seed=6)


def backward(lib, m, k, n, dtype, act, xk, pk, dyt, dxt, dwt, extra=0, seed=0, which="xwb"):
    rng, x, w = make(lib, m, k, n, dtype, seed, extra)
    x = Operand(lib, m, k, xk, torch.from_numpy(x.values()), extra)
    z = Operand(lib, m, n, pk, torch.from_numpy(1.5 * rng.normal(size=(m, n))), extra) if pk else None
    dy = Operand(lib, m, n, dyt, torch.from_numpy(rng.normal(size=(m, n))), extra)
    dx = Operand(lib, m, k, dxt, extra=extra) if "x" in which else None
    dw = Operand(lib, n, k, dwt, extra=extra) if "w" in which else None
    db = torch.full((n + 4,), 7.0, device="cuda")
    need = lib.st_linear_workspace_bytes(m, k, n, dtype, backward=True)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    lib.st_linear_backward(x.t, w.t, dy.t, dx.t if dx else None, dw.t if dw else None, db[:n] if "b" in which else None,
                           act=act, pre=z.t if z else None, workspace=ws[:need])
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0x5A).all()) and bool((db[n:] == 7.0).all())
    xv, wv, dv = x.values(), w.values(), dy.values()
    wdx, wdw, wdb = mlp.linear_backward(xv, wv, dv, act, z.values() if z else None)
    # p in fp32: a slope is a sum of terms up to 1.2 that may cancel (Phi(z) + z phi(z),
    # s + s z (1 - s)), each a few 2^-24 off by its exponential, reciprocal and
    # polynomial steps: 2^-20 in all, absolute.  Then rounded to bf16 where the
    # products are bf16 and p is not so already
    p = np.abs(dv) * (1.0 if act == "none" else np.abs(mlp.slope(z.values(), act)))
    e = np.abs(dv) * (2.0 ** -20 if act in ("gelu", "silu") else 0)
    half = 2.0 ** -8 * 1.001 if dtype == "bf16" and (act != "none" or dyt == "f32") else 0

    def tol(count, mat, left):
        both = (lambda q: q @ mat) if left else (lambda q: q.T @ mat)
        return both((half + sums(count)) * (p + e) + e)

    if dx:
        dx.check_guards()
        within("dx", dx.values(), wdx, tol(n, np.abs(wv), True) + rounding(wdx, dxt) * 1.01)
    if dw:
        dw.check_guards()
        within("dw", dw.values(), wdw, tol(m, np.abs(xv), False) + rounding(wdw, dwt) * 1.01)
    if "b" in which:
        within("dbias", npy(db[:n]), wdb, (sums(m) * (p + e) + e).sum(0))
    else:
        assert bool((db == 7.0).all())


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("extra", [0, 40])
def test_gradients(gpu_lib, m, k, n, dtype, extra):
    say(f"linear backward {m}x{k}x{n} {dtype} extra {extra}")
    backward(gpu_lib, m, k, n, dtype, "none", dtype, "", dtype, dtype, "f32", extra, seed=m + k + n)
    backward(gpu_lib, m, k, n, dtype, "gelu", "mx8", "mx8", dtype, "f32", dtype, extra, seed=m + k)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("dtype,dy", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("xk", ["same", "mx8"])
@pytest.mark.parametrize("pk", ["f32", "bf16", "mx8"])
def test_gradient_forms(gpu_lib, act, dtype, dy, xk, pk):
    say(f"linear backward {act} {dtype} {dy} {xk} {pk}")
    backward(gpu_lib, 90, 72, 110, dtype, act, dtype if xk == "same" else xk, pk if act != "none" else "", dy, "f32", "f32", seed=7)


@pytest.mark.parametrize("which", ["x", "w", "b", "xb", "wb", "xw"])
def test_gradients_apart(gpu_lib, which):
    backward(gpu_lib, 70, 64, 48, "bf16", "silu", "bf16", "bf16", "bf16", "bf16", "f32", which=which)
    backward(gpu_lib, 70, 64, 48, "bf16", "none", "bf16", "", "bf16", "bf16", "f32", which=which)


@pytest.mark.parametrize("m,k,n", [(3000, 136, 264), (8200, 64, 40), (600, 1032, 520)])
def test_long_gradients(gpu_lib, m, k, n):
    say(f"linear backward {m}x{k}x{n}")
    backward(gpu_lib, m, k, n, "bf16", "relu", "bf16", "bf16", "bf16", "bf16", "f32", seed=8)
    backward(gpu_lib, m, k, n, "f32", "none", "f32", "", "f32", "f32", "f32", seed=9)


def test_no_rows(gpu_lib):
    """Nothing forward; dw and dbias are cleared."""
    w = torch.ones(24, 40, dtype=torch.bfloat16, device="cuda")
    x, y = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    gpu_lib.st_linear(x, w, None, y)
    dw, db = torch.ones(24, 40, device="cuda"), torch.ones(24, device="cuda")
    gpu_lib.st_linear_backward(x, w, y, torch.empty_like(x), dw, db, workspace=None)
    assert bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mx8"])
def test_what_lies_behind_a_row_has_no_part(gpu_lib, dtype):
    """NaN between the rows and behind the operands: none of it reaches a result."""
    for m, k, n in ((5, 44, 9), (70, 100, 130)):
        rng, x, w = make(gpu_lib, m, k, n, dtype, 11, 40)
        want = mlp.linear(x.values(), w.values())[0]
        for o in (x, w):
            keep = o.t.codes[:, :k].clone() if dtype == "mx8" else o.t.clone()
            if dtype == "mx8":
                o.store.fill_(0x7F)
                o.store[:o.rows, :k] = keep
                blocks = -(-k // 32)
                keep = o.t.scales[:, :blocks].clone()
                o.sstore.fill_(0xFF)
                o.sstore[:o.rows, :blocks] = keep
            else:
                o.store.fill_(math.nan)
                o.t.copy_(keep)
        y = torch.empty(m, n, device="cuda")
        ws = torch.full((max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, dtype)),), 0xFF, dtype=torch.uint8, device="cuda")
        gpu_lib.st_linear(x.t, w.t, None, y, workspace=ws)
        within("y", npy(y), want, sums(k) * (np.abs(x.values()) @ np.abs(w.values()).T))


def test_special_values_stay_in_their_rows(gpu_lib):
    """A NaN in a token reaches that token alone, an infinite residual its element."""
    m, k, n = 140, 64, 96
    rng, x, w = make(gpu_lib, m, k, n, "bf16")
    x.t[17, 3] = math.nan
    res = torch.zeros(m, n, device="cuda")
    res[20, 5] = math.inf
    y = torch.empty(m, n, device="cuda")
    ws = torch.empty(max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, "bf16")), dtype=torch.uint8, device="cuda")
    gpu_lib.st_linear(x.t, w.t, None, y, act="gelu", residual=res, workspace=ws)
    bad = ~torch.isfinite(y)
    assert bool(bad[17].all()) and bool(bad[20, 5]) and int(bad.sum()) == n + 1


@pytest.mark.parametrize("act,lo,hi", [("relu", 0.0, math.inf), ("gelu", 0.0, math.inf), ("silu", 0.0, math.inf)])
def test_activations_far_out(gpu_lib, act, lo, hi):
    """Large arguments and infinities take the limits, value and slope; NaN stays."""
    v = torch.tensor([[-math.inf, -1e30, -200.0, -50.0, 50.0, 200.0, 1e30, math.inf, math.nan, 0.0, -0.0, 1e-30]], device="cuda")
    c = v.shape[1]
    # through the bias: x w^T = 0
    x, w = torch.zeros(1, 4, device="cuda"), torch.zeros(c, 4, device="cuda")
    y = torch.empty(1, c, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    gpu_lib.st_linear(x, w, v[0].contiguous(), y, act=act, workspace=ws)
    got = y[0].cpu()
    assert bool((got[:3] == 0).all()) and abs(float(got[3])) < 1e-18 and bool((got[4:8] == v[0, 4:8].cpu()).all())
    assert math.isnan(got[8]) and bool((got[9:11] == 0).all()) and abs(float(got[11])) <= float(v[0, 11])
    db = torch.empty(c, device="cuda")
    gpu_lib.st_linear_backward(x, w, torch.ones(1, c, device="cuda"), None, None, db, act=act, pre=v, workspace=ws)
    d = db.cpu()
    assert float(d[:4].abs().max()) < 1e-18 and bool((d[4:8] == 1).all())
    assert act == "relu" or math.isnan(d[8])


def test_in_place_residual_and_views(gpu_lib):
    """y onto the residual's own buffer; x and y as column views of wider buffers."""
    m, k, n = 100, 64, 128
    rng, x, w = make(gpu_lib, m, k, n, "bf16")
    stream = torch.from_numpy(rng.normal(size=(m, n))).float().cuda()
    ws = torch.empty(max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, "bf16")), dtype=torch.uint8, device="cuda")
    apart = torch.empty_like(stream)
    gpu_lib.st_linear(x.t, w.t, None, apart, residual=stream, workspace=ws)
    gpu_lib.st_linear(x.t, w.t, None, stream, residual=stream, workspace=ws)
    assert torch.equal(apart, stream)
    wide = torch.zeros(m, 2 * k + n, dtype=torch.bfloat16, device="cuda")
    wide[:, k:2 * k].copy_(x.t)
    gpu_lib.st_linear(wide[:, k:2 * k], w.t, None, wide[:, 2 * k:], workspace=ws)
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    gpu_lib.st_linear(x.t, w.t, None, y, workspace=ws)
    assert torch.equal(wide[:, 2 * k:], y) and bool((wide[:, :k] == 0).all())


def test_rows_past_32_bits(gpu_lib):
    """Operands of more than 2^32 bytes: rows at both ends, and a weight gradient
    over them."""
    m, k, n = (1 << 21) + 300, 1032, 40
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(12)
    tail = torch.from_numpy(rng.normal(size=(400, k))).to(torch.bfloat16).cuda()
    x[-400:].copy_(tail)
    w = torch.from_numpy(rng.normal(size=(n, k)) / 32).to(torch.bfloat16).cuda()
    y = torch.empty(m, n, device="cuda")
    ws = torch.empty(max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, "bf16", backward=True)), dtype=torch.uint8, device="cuda")
    gpu_lib.st_linear(x, w, None, y, workspace=ws)
    want = mlp.linear(npy(tail), npy(w))[0]
    within("y", npy(y[-400:]), want, sums(k) * (np.abs(npy(tail)) @ np.abs(npy(w)).T))
    assert bool((y[:-400] == 0).all())
    dy = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    dy[-400:] = torch.from_numpy(rng.normal(size=(400, n))).to(torch.bfloat16).cuda()
    dy[:1000] = 1.0                                       # (their x is zero)
    dx, dw, db = torch.empty_like(x), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    gpu_lib.st_linear_backward(x, w, dy, dx, dw, db, workspace=ws)
    d = npy(dy[-400:])
    within("dw", npy(dw), d.T @ npy(tail), sums(400) * 2 * (np.abs(d).T @ np.abs(npy(tail))))
    within("dx", npy(dx[-400:]), d @ npy(w), sums(n) * (np.abs(d) @ np.abs(npy(w))) + rounding(d @ npy(w), "bf16") * 1.01)
    within("dbias", npy(db), d.sum(0) + 1000, sums(1400) * (np.abs(d).sum(0) + 1000))


def test_same_bits_twice(gpu_lib):
    m, k, n = 1000, 520, 264
    rng, x, w = make(gpu_lib, m, k, n, "bf16")
    dy = torch.from_numpy(rng.normal(size=(m, n))).to(torch.bfloat16).cuda()
    ws = torch.empty(gpu_lib.st_linear_workspace_bytes(m, k, n, "bf16", backward=True), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(3):
        ws.fill_(0xFF)
        dx, dw, db = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
        gpu_lib.st_linear_backward(x.t, w.t, dy, dx, dw, db, workspace=ws)
        got.append((dx, dw, db))
    for a, b, c in zip(*got):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mx8"])
@pytest.mark.parametrize("k", [40, 64, 136, 200, 520, 1000])
@pytest.mark.parametrize("y,pre,res", [("bf16", "", ""), ("f32", "", ""), ("bf16", "mx8", "f32"), ("mx8", "", "bf16"), ("f32", "bf16", "f32")])
def test_many_tiles_of_whole_numbers(gpu_lib, dtype, k, y, pre, res):
    """Several tiles a workgroup, whole ones and ragged ones, of one stage and more,
    bit for bit: whole numbers up to 3, whose sums (below 9 * 1000 + 3 + 3) are exact in fp32
    and in the 8-bit instructions (products of up to 4 bits, sums of eight in 7)."""
    say(f"linear whole numbers k {k} {dtype} y {y} pre {pre} res {res}")
    m, n = 10247, 2312
    gen = torch.Generator(device="cuda").manual_seed(k)
    draw = lambda *s: torch.randint(-3, 4, s, generator=gen, device="cuda").float()  # noqa: E731
    xf, wf, b, r = draw(m, k), draw(n, k), draw(n), draw(m, n)

    def held(t, d):
        if d == "mx8":
            o = gpu_lib.mx8_empty(*t.shape)
            gpu_lib.st_mx8_store(t, o)
            return o
        return t.to(TORCH[d])

    def blank(d):
        return None if not d else gpu_lib.mx8_empty(m, n) if d == "mx8" else torch.full((m, n), 99.0, device="cuda").to(TORCH[d])

    yo, po = blank(y), blank(pre)
    ws = torch.empty(max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, dtype)), dtype=torch.uint8, device="cuda")
    gpu_lib.st_linear(held(xf, dtype), held(wf, dtype), b, yo, act="relu", residual=held(r, res) if res else None, pre=po, workspace=ws)
    z = (xf.double() @ wf.double().t() + b.double()).float()
    want = torch.relu(z) + (r if res else 0)
    for got, value, d in ((yo, want, y), (po, z, pre)):
        if d == "mx8":
            exact = held(value, "mx8")
            blocks = -(-n // 32)
            assert torch.equal(got.codes[:, :n], exact.codes[:, :n]) and torch.equal(got.scales[:, :blocks], exact.scales[:, :blocks])
        elif d:
            assert torch.equal(got, value.to(TORCH[d]))


def test_two_graphs_of_one_workspace(gpu_lib):
    """Captured calls that share a workspace, replayed in turns with eager work between."""
    m, k, n = 96, 4104, 264                               # split and joined, rows copied whole
    rng = np.random.default_rng(13)
    x = [torch.from_numpy(rng.normal(size=(m, k))).bfloat16().cuda() for _ in range(2)]
    w = torch.from_numpy(rng.normal(size=(n, k)) / 64).bfloat16().cuda()
    dy = torch.from_numpy(rng.normal(size=(m, n))).bfloat16().cuda()
    need = max(gpu_lib.st_linear_workspace_bytes(m, k, n, "bf16"), gpu_lib.st_linear_workspace_bytes(m, k, n, "bf16", backward=True))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def outputs():
        return [torch.zeros(m, n, device="cuda"), torch.zeros(m, k, device="cuda"), torch.zeros(n, k, device="cuda"), torch.zeros(n, device="cuda")]

    def run(i, o):
        gpu_lib.st_linear(x[i], w, None, o[0], act="silu", workspace=ws)
        gpu_lib.st_linear_backward(x[i], w, dy, *o[1:], workspace=ws)

    want, outs, graphs = [outputs() for _ in range(2)], [outputs() for _ in range(2)], []
    for i in range(2):
        run(i, want[i])
    torch.cuda.synchronize()
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            run(i, outs[i])
    for turn in range(3):
        for i in range(2):
            for t in outs[i]:
                t.zero_()
            ws.fill_(0xFF)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i])), f"turn {turn} graph {i}"
