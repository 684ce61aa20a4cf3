"""Rotary positions with several axes, and the positions of a sharded volume's
cells, against the fp64 definition.

Tolerance, element by element: the angle is right to 2^-23 turns and cos and sin
to a few 2^-24, the rotation is two products and a sum in fp32: 2^-20 of
|u| + |v|; a bf16 output adds its rounding, 2^-8 of its value.
"""
import math

import numpy as np
import pytest
import torch

from helpers import say
from oracle import tokens

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def check(got, x, pos, dims, **kw):
    want = tokens.rope(x.double().cpu().numpy(), pos.cpu().numpy(), dims, **kw)
    size = np.abs(x.double().cpu().numpy())
    bound = size + size.max(-1, keepdims=True)            # |u| + |v| of any pair
    tol = 2.0 ** -20 * bound + (2.0 ** -8 * np.abs(want) * 1.001 if got.dtype == torch.bfloat16 else 0)
    off = np.abs(got.double().cpu().numpy() - want)
    assert np.all(off <= tol), f"off {off.max()}, over by {np.max(off - tol)}"


@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("xt,ot", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("dims,dim,heads,rotated", [
    ([32, 32], 64, 4, 4), ([16, 24, 24], 64, 6, 4), ([128], 128, 3, 1), ([2, 6], 12, 2, 2), ([20, 18, 22], 64, 5, 5),
    ([0, 40], 72, 1, 1), ([10, 14], 40, 3, 0), ([80, 80, 96], 256, 2, 2)])
def test_rotation(gpu_lib, dims, dim, heads, rotated, xt, ot, pairs):
    say(f"rope {dims} of {dim}, {rotated} of {heads} heads, {xt}->{ot} {pairs}")
    rng = np.random.default_rng(0)
    t = 77
    x = torch.from_numpy(rng.normal(size=(t, heads, dim))).to(TORCH[xt]).cuda()
    pos = torch.from_numpy(rng.integers(0, 4096, size=(t, len(dims)))).to(torch.int32).cuda()
    kw = dict(pairs=pairs, rotated_heads=rotated)
    for inverse in (False, True):
        out = torch.full((t, heads, dim), 7.0, dtype=TORCH[ot], device="cuda")
        gpu_lib.st_rope_axes(x, pos, dims, out, inverse=inverse, **kw)
        check(out, x, pos, dims, inverse=inverse, **kw)
        if xt == ot:
            same = x.clone()
            gpu_lib.st_rope_axes(same, pos, dims, same, inverse=inverse, **kw)
            assert torch.equal(same, out)


@pytest.mark.parametrize("tokens_", [0, 1, 2, 513, 5000])
def test_token_counts_and_far_positions(gpu_lib, tokens_):
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.normal(size=(tokens_, 2, 64))).float().cuda()
    pos = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, size=(tokens_, 3))).to(torch.int32).cuda()
    out = torch.empty_like(x)
    gpu_lib.st_rope_axes(x, pos, [16, 24, 24], out)
    if tokens_:
        check(out, x, pos, [16, 24, 24])


def test_views(gpu_lib):
    """A joint projection as input, heads outermost as output; what lies between
    the rows stays."""
    rng = np.random.default_rng(2)
    b = torch.from_numpy(rng.normal(size=(50, 9, 72))).bfloat16().cuda()
    x = b[:, 2:7, :64]
    ob = torch.full((5, 50, 80), 3.0, dtype=torch.bfloat16, device="cuda")
    out = ob[:, :, :64].transpose(0, 1)
    pos = torch.from_numpy(rng.integers(0, 99, size=(50, 2))).to(torch.int32).cuda()
    gpu_lib.st_rope_axes(x, pos, [32, 32], out)
    check(out, x, pos, [32, 32])
    assert bool((ob[:, :, 64:] == 3.0).all())


def test_offsets_past_32_bits(gpu_lib):
    """2.3e9 values: the last tokens are those of a small call."""
    t = 140000
    x = torch.empty(t, 64, 256, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    pos = torch.arange(2 * t, dtype=torch.int32, device="cuda").view(t, 2)
    want = x[-30:].clone()
    gpu_lib.st_rope_axes(want, pos[-30:].clone(), [128, 128], want)
    gpu_lib.st_rope_axes(x, pos, [128, 128], x)
    assert torch.equal(x[-30:], want)


def test_special_values_outside_the_rotation(gpu_lib):
    """Copied channels and heads keep NaN, infinities and the sign of zero."""
    x = torch.randn(6, 3, 64, device="cuda")
    x[:, :, 40:] = torch.tensor([math.inf, -math.inf, math.nan, -0.0], device="cuda").repeat(6)
    x[:, 2] = math.inf
    pos = torch.arange(12, dtype=torch.int32, device="cuda").view(6, 2)
    out = torch.empty_like(x)
    gpu_lib.st_rope_axes(x, pos, [20, 20], out, rotated_heads=2)
    assert torch.equal(out[:, :, 40:].view(torch.int32), x[:, :, 40:].contiguous().view(torch.int32))
    assert torch.equal(out[:, 2], x[:, 2]) and bool(torch.isfinite(out[:, :2, :40]).all())


def test_positions_of_sharded_cells(gpu_lib):
    for spatial, sizes, halo in (((7, 9), ((3, 4), (5, 4)), 1), ((4, 5, 6), ((4,), (2, 3), (1, 5)), 0)):
        nd = len(spatial)
        plan = gpu_lib.st_plan_shards(nd, 2, 8, spatial, sizes, [halo] * nd, "f32")
        infos = [plan.shard_info(i) for i in range(plan.num_shards)]
        bufs = [torch.full((2, *inf["extent"], nd), -1, dtype=torch.int32, device="cuda") for inf in infos]
        gpu_lib.st_plan_positions(plan, bufs)
        for inf, b in zip(infos, bufs):
            grid = torch.stack(torch.meshgrid(*[torch.arange(o, o + e) for o, e in zip(inf["offset"], inf["extent"])],
                                              indexing="ij"), -1).to(torch.int32)
            assert torch.equal(b.cpu(), grid.expand(2, *grid.shape))


def test_refusals_on_the_gpu(gpu_lib):
    x = torch.zeros(4, 2, 64, device="cuda")
    pos = torch.zeros(4, 2, dtype=torch.int32, device="cuda")

    def status(*a, **kw):
        with pytest.raises(gpu_lib.ShardConvError) as e:
            gpu_lib.st_rope_axes(*a, **kw)
        return e.value.status

    assert status(x, pos, [3, 4], x) == 2                  # odd width
    assert status(x, pos, [40, 40], x) == 2                # wider than the head
    assert status(x, pos, [32, 32], x, base=1.0) == 1
    assert status(x, pos, [32, 32], x, pairs="thirds") == 1
    assert status(x, pos, [32, 32], x, rotated_heads=3) == 1
    assert status(x, pos.long(), [32, 32], x) == 1
    assert status(x, pos[:3], [32, 32], x) == 2
    assert status(x, pos, [32, 32], x[:3]) == 2
    assert status(x, pos, [], x) == 4
    assert status(x, pos, [32, 32], x.double()) == 1
    assert status(x, pos, [32, 32], torch.zeros(1, 1, 64, device="cuda").expand(4, 2, 64)) == 2


def test_positions_of_more_cells_than_one_launch_holds(gpu_lib):
    """4.5e9 cells, over 2^32 threads: three samples in three shards of 5e8 columns."""
    w = [500000001, 500000000, 499999999]
    plan = gpu_lib.st_plan_shards(2, 3, 8, (1, sum(w)), ((1,), w), (0, 0), "bf16")
    bufs = [torch.full((3, 1, n, 2), -1, dtype=torch.int32, device="cuda") for n in w]
    gpu_lib.st_plan_positions(plan, bufs)
    for i, b in enumerate(bufs):
        assert not b[..., 0].any()
        want = torch.arange(sum(w[:i]), sum(w[:i + 1]), dtype=torch.int32, device="cuda")
        assert all(torch.equal(b[n, 0, :, 1], want) for n in range(3))


@pytest.mark.parametrize("tokens_,heads", [(2 ** 31 - 1, 1), ((1 << 24) + 3, 1025)])
def test_most_tokens(gpu_lib, tokens_, heads):
    """The most tokens that a call takes, whose number rounded up to whole
    workgroups passes 31 bits; and 2^24 workgroups, one more than a launch takes."""
    x = torch.empty(tokens_, heads, 2, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    pos = torch.arange(tokens_, dtype=torch.int32, device="cuda").view(-1, 1)
    ends = [slice(0, 30), slice((1 << 24) - 20, (1 << 24) + 2), slice(tokens_ - 30, tokens_)]
    want = [x[e].clone() for e in ends]
    for w, e in zip(want, ends):
        gpu_lib.st_rope_axes(w, pos[e].clone(), [2], w)
    gpu_lib.st_rope_axes(x, pos, [2], x)
    assert all(torch.equal(x[e], w) for e, w in zip(ends, want))


def test_positions_of_another_number_of_axes(gpu_lib):
    """Three axes' positions with two sections are refused, not read across rows;
    grids and flat buffers of the right number pass."""
    x = torch.randn(6, 2, 64, device="cuda")
    pos = torch.arange(18, dtype=torch.int32, device="cuda")
    with pytest.raises(gpu_lib.ShardConvError) as e:
        gpu_lib.st_rope_axes(x, pos.view(6, 3), [32, 32], x.clone())
    assert e.value.status == 2
    outs = [torch.empty_like(x) for _ in range(3)]
    for o, p in zip(outs, (pos.view(6, 3), pos.view(2, 3, 3), pos)):
        gpu_lib.st_rope_axes(x, p, [16, 24, 24], o)
    check(outs[0], x, pos.view(6, 3), [16, 24, 24])
    assert torch.equal(outs[1], outs[0]) and torch.equal(outs[2], outs[0])


@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_one_token_or_one_head_has_no_stride(gpu_lib, pairs):
    """Whatever stride a view names for it, odd or other than the output's."""
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.normal(size=(4, 4, 64))).bfloat16().cuda()
    pos = torch.from_numpy(rng.integers(0, 99, size=(4, 2))).to(torch.int32).cuda()
    for tokens_, heads, strides in ((1, 4, (65, 64, 1)), (4, 1, (256, 3, 1)), (1, 1, (7, 9, 1))):
        p, src = pos[:tokens_].contiguous(), x[:tokens_, :heads].contiguous()
        want = torch.empty_like(src)
        gpu_lib.st_rope_axes(src, p, [32, 32], want, pairs=pairs)
        check(want, src, p, [32, 32], pairs=pairs)
        v = x.clone().as_strided((tokens_, heads, 64), strides)
        same = v.as_strided((tokens_, heads, 64), (256, 64, 1))
        out = torch.empty_like(want)
        gpu_lib.st_rope_axes(v, p, [32, 32], out, pairs=pairs)
        assert torch.equal(out, want)
        gpu_lib.st_rope_axes(v, p, [32, 32], same, pairs=pairs)   # in place, under other strides
        assert torch.equal(same, want)
