"""Matrix products in every tile that there is, over several tiles a workgroup, and
their 8-bit operands and outputs bit for bit."""
import math

import numpy as np
import pytest
import torch

from helpers import say
from linear_tiles import TILES
from mlp_helpers import TORCH

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n", [(5, 40), (40, 130), (300, 200), (1100, 600)])
@pytest.mark.parametrize("k", [40, 128, 200, 1000, 4104])
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_scales_that_end_a_buffer(gpu_lib, m, n, k, y):
    """Scales as the last columns of a wider buffer, whose last byte is theirs: the
    bits of scales that lie by themselves."""
    say(f"linear {m}x{k}x{n} mx8, y {y}, scales in the last columns of a buffer")
    rng = np.random.default_rng(m + n + k)
    own, ends = [], []
    for rows, size in ((m, 1.0), (n, 1 / math.sqrt(k))):
        o = gpu_lib.mx8_empty(rows, k)
        o.scales.zero_()
        gpu_lib.st_mx8_store(torch.from_numpy(np.float32(size * rng.normal(size=(rows, k)))).cuda(), o)
        words = o.scales.shape[1]
        wide = torch.full((rows, 16 + words), 0xFF, dtype=torch.uint8, device="cuda")
        wide[:, 16:] = o.scales
        own.append(o)
        ends.append(gpu_lib.Mx8(o.codes, wide[:, 16:], k))
    got = []
    ws = torch.empty(max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, "mx8")), dtype=torch.uint8, device="cuda")
    for x, w in (own, ends):
        out = torch.full((m, n), math.nan, device="cuda").to(torch.float32 if y == "f32" else torch.bfloat16)
        gpu_lib.st_linear(x, w, None, out, workspace=ws)
        got.append(out)
    assert bool(torch.isfinite(got[0]).all()) and torch.equal(*got)


# ------------------------------------------------------- whole numbers, every tile
#
# Values up to 3 and contractions up to 29468 have sums below 9 * 29468 + 6 < 2^24: exact
# in fp32 in any order, and in the 8-bit instructions (products of up to 4 bits, sums of
# eight in 7).  So every output has the bits of the 64-bit sums rounded once.

def numbers(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randint(-3, 4, s, generator=gen, device="cuda").float()


def held(lib, t, dtype):
    if dtype == "mx8":
        o = lib.mx8_empty(*t.shape)
        lib.st_mx8_store(t, o)
        return o
    return t.to(TORCH[dtype])


def blank(lib, dtype, *shape):
    """An output with guard bytes behind its last row."""
    if dtype == "mx8":
        return lib.mx8_empty(*shape), None
    t = torch.full((shape[0] + 1, shape[1]), 99.0, device="cuda").to(TORCH[dtype])
    return t[:-1], t[-1]


def same(lib, out, want, dtype):
    got, behind = out
    if dtype == "mx8":
        exact = held(lib, want, "mx8")
        blocks = -(-want.shape[1] // 32)
        return torch.equal(got.codes[:, :want.shape[1]], exact.codes[:, :want.shape[1]]) and torch.equal(got.scales[:, :blocks], exact.scales[:, :blocks])
    return torch.equal(got, want.to(TORCH[dtype])) and bool((behind == 99.0).all())


def sizes_of(*products):
    return [t for t in TILES if t[0] in products]


@pytest.mark.parametrize("product,dtype,m,k,n,widened,tile,stages", sizes_of("y"))
def test_forward_in_every_tile(gpu_lib, product, dtype, m, k, n, widened, tile, stages):
    """With nothing but a bias (outputs in bf16 and fp32), and with everything there is."""
    draw = numbers(m + k + n)
    xf, wf, b, r = draw(m, k), draw(n, k), draw(n), draw(m, n)
    x, w, res = held(gpu_lib, xf, dtype), held(gpu_lib, wf, dtype), held(gpu_lib, r, "f32")
    z = (xf.double() @ wf.double().t() + b.double()).float()
    want = torch.relu(z) + r
    ws = torch.empty(max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, dtype)), dtype=torch.uint8, device="cuda")
    # (of 8-bit operands an output that is no bf16 takes the widened products)
    if dtype != "mx8":
        forms = [("none", "bf16", "", False), ("none", "f32", "", False), ("relu", "bf16", "mx8", True), ("relu", "f32", "bf16", False)]
    elif widened:
        forms = [("none", "f32", "", False), ("none", "mx8", "", False), ("relu", "mx8", "bf16", True), ("relu", "bf16", "mx8", False)]
    else:
        forms = [("none", "bf16", "", False), ("relu", "bf16", "bf16", True), ("relu", "bf16", "", False)]
    for act, y, pre, added in forms:
        say(f"y {m}x{k}x{n} {dtype} tiles of {tile}, {stages} stages: {act} y {y} pre {pre} residual {added}")
        yo, po = blank(gpu_lib, y, m, n), blank(gpu_lib, pre, m, n) if pre else (None, None)
        gpu_lib.st_linear(x, w, b, yo[0], act=act, residual=res if added else None, pre=po[0], workspace=ws)
        assert same(gpu_lib, yo, z if act == "none" else want if added else torch.relu(z), y)
        if pre:
            assert same(gpu_lib, po, z, pre)


@pytest.mark.parametrize("product,dtype,m,k,n,widened,tile,stages", sizes_of("dx", "dw"))
def test_gradients_in_every_tile(gpu_lib, product, dtype, m, k, n, widened, tile, stages):
    """dx or dw alone: of dy as it is, and of p formed from an activation, an fp32 dy and
    an input and a pre-activation kept in 8 bits."""
    draw = numbers(m + k + n)
    xf, wf, dyf, pf = draw(m, k), draw(n, k), draw(m, n), draw(m, n)
    w = held(gpu_lib, wf, dtype)
    ws = torch.empty(gpu_lib.st_linear_workspace_bytes(m, k, n, dtype, backward=True), dtype=torch.uint8, device="cuda")
    for act, xk, dyt, out in (("none", dtype, dtype, "f32"), ("none", dtype, dtype, "bf16"), ("relu", "mx8", "f32", "f32")):
        say(f"{product} {m}x{k}x{n} {dtype} tiles of {tile}, {stages} stages: {act} x {xk} dy {dyt} out {out}")
        p = dyf * (pf > 0) if act == "relu" else dyf
        dx, dw = (blank(gpu_lib, out, m, k), (None, None)) if product == "dx" else ((None, None), blank(gpu_lib, out, n, k))
        db = torch.full((n,), 99.0, device="cuda")
        gpu_lib.st_linear_backward(held(gpu_lib, xf, xk), w, held(gpu_lib, dyf, dyt), dx[0], dw[0], db, act=act,
                                   pre=held(gpu_lib, pf, "mx8") if act == "relu" else None, workspace=ws)
        if product == "dx":
            assert same(gpu_lib, dx, (p.double() @ wf.double()).float(), out)
        else:
            assert same(gpu_lib, dw, (p.double().t().contiguous() @ xf.double()).float(), out)
        assert torch.equal(db, p.double().sum(0).float())


# ----------------------------------------- 8-bit operands: what is rounded to 8 bits

@pytest.mark.parametrize("m,k,n", [(1, 2048, 520), (7, 200, 96), (33, 8192, 256), (64, 1000, 300),      # few rows, whole and split
                                   (300, 9000, 260), (150, 128, 200), (8448, 1000, 2304), (9000, 144, 2304)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_eight_bit_outputs_are_the_fp32_outputs_rounded(gpu_lib, m, k, n, act):
    """8-bit outputs of 8-bit operands come from the sums that an fp32 output shows, not
    from those that the 8-bit instructions cut: codes and scales are st_mx8_store's of the
    fp32 output, of y and of the pre-activation, whichever of them is in 8 bits."""
    say(f"linear {m}x{k}x{n} mx8 {act}: 8-bit outputs")
    gen = torch.Generator(device="cuda").manual_seed(m + k + n)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, w = held(gpu_lib, normal(m, k) * (0.25 + 1.5 * torch.rand(k, generator=gen, device="cuda")), "mx8"), held(gpu_lib, normal(n, k) / math.sqrt(k), "mx8")
    b = 0.2 * normal(n)
    ws = torch.empty(max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, "mx8")), dtype=torch.uint8, device="cuda")

    def run(y, pre):
        yo, po = blank(gpu_lib, y, m, n), blank(gpu_lib, pre, m, n) if pre else (None, None)
        gpu_lib.st_linear(x, w, b, yo[0], act=act, pre=po[0], workspace=ws)
        return yo, po

    (yf, _), (zf, _) = run("f32", "f32")
    for y, pre in (("mx8", ""), ("mx8", "bf16"), ("bf16", "mx8"), ("mx8", "mx8"), ("f32", "mx8")):
        yo, po = run(y, pre)
        assert same(gpu_lib, yo, yf, y), f"y {y} pre {pre}"
        assert not pre or same(gpu_lib, po, zf, pre), f"pre {pre} y {y}"


@pytest.mark.parametrize("m,k,n", [(7, 200, 96), (40, 8192, 260), (300, 9000, 260), (8449, 1000, 2304), (2716, 257, 2299)])
@pytest.mark.parametrize("dtype", ["bf16", "mx8", "f32"])
@pytest.mark.parametrize("stream", ["f32", "bf16"])
def test_output_in_the_residuals_place(gpu_lib, m, k, n, dtype, stream):
    """Few rows, split and joined sums, several tiles a workgroup: the bits of an output
    of its own."""
    say(f"linear {m}x{k}x{n} {dtype} onto its {stream} residual")
    gen = torch.Generator(device="cuda").manual_seed(m)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, w, r = held(gpu_lib, normal(m, k), dtype), held(gpu_lib, normal(n, k) / math.sqrt(k), dtype), normal(m, n).to(TORCH[stream])
    ws = torch.empty(max(16, gpu_lib.st_linear_workspace_bytes(m, k, n, dtype)), dtype=torch.uint8, device="cuda")
    apart = torch.empty_like(r)
    gpu_lib.st_linear(x, w, None, apart, act="silu", residual=r, workspace=ws)
    gpu_lib.st_linear(x, w, None, r, act="silu", residual=r, workspace=ws)
    assert bool(torch.isfinite(apart).all()) and torch.equal(apart, r)
