"""The attention branch (layer norm, 1x1 convs, rotary positions, attention and
their gradients) on a sharded volume against its fp64 definition, and against
the unsharded run.

Tolerance: every bf16 rounding on the way (the normed cells, q, k, v, the
weights p, the attended values, and their gradients: at most 8 in a row) is off
by 2^-9 of its value in the mean square; independent errors add in squares and
each step's gain is about one: sqrt(8) 2^-9 = 0.6%, held to 2% of the norm.
"""
import numpy as np
import pytest
import torch

from helpers import say
from oracle import tokens

pytestmark = pytest.mark.gpu


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().double().numpy()


def reference(layer, x, pos, w_qkv, w_out, gamma, beta, dy, lens):
    t, h, hk, d = len(x), layer.heads, layer.kv_heads, layer.head_dim
    n, _, _ = tokens.layer_norm(x, gamma, beta, layer.eps)
    qkv = (n @ w_qkv.T).reshape(t, h + 2 * hk, d)
    turn = dict(axis_dims=layer.axis_dims, base=layer.base, rotated_heads=h + hk)
    r = tokens.rope(qkv, pos, **turn)
    q, k, v = r[:, :h], r[:, h:h + hk], r[:, h + hk:]
    dout = (dy @ w_out).reshape(t, h, d)
    a = tokens.attention(q, k, v, lens, lens, layer.scale, False, dout)
    out = a["out"].reshape(t, h * d)
    dr = np.concatenate([a["dq"], a["dk"], a["dv"]], 1)
    dqkv = tokens.rope(dr, pos, inverse=True, **turn).reshape(t, -1)
    dx, dg, db = tokens.layer_norm_backward(x, dqkv @ w_qkv, gamma, layer.eps)
    return {"y": out @ w_out.T, "dx": dx, "dgamma": dg, "dbeta": db, "dw_qkv": dqkv.T @ n, "dw_out": dy.T @ out}


def off(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("spatial,shards,batch,channels,heads,kv_heads,dim", [
    ((9, 14), ((4, 5), (14,)), 1, 32, 4, 2, 16),          # an image in two row shards
    ((4, 6, 10), ((4,), (6,), (7, 3)), 1, 48, 3, 1, 32),  # a volume cut along its width
    ((8, 8), ((8,), (8,)), 3, 64, 4, 4, 16),              # three samples
])
def test_branch(gpu_lib, spatial, shards, batch, channels, heads, kv_heads, dim):
    from halo_sharded_conv_amd.attention_layer import ShardedAttention
    say(f"attention branch {spatial} {shards} C={channels} {heads}/{kv_heads} x {dim}")
    rng = np.random.default_rng(0)
    layer = ShardedAttention(spatial, shards, channels, heads, kv_heads, dim, batch=batch)
    t = layer.tokens
    x = np.float32(rng.normal(size=(t, channels)) + 0.3)
    w_qkv = bf16(rng.normal(size=(layer.joint_width, channels)) / np.sqrt(channels))
    w_out = bf16(rng.normal(size=(channels, layer.width)) / np.sqrt(layer.width))
    gamma, beta = np.float32(1 + 0.2 * rng.normal(size=channels)), np.float32(0.2 * rng.normal(size=channels))
    dy = bf16(rng.normal(size=(t, channels)))
    layer.set_weights(w_qkv, w_out, gamma, beta)
    xd, dyd = torch.from_numpy(x).cuda(), torch.from_numpy(dy).bfloat16().cuda()
    y = layer.forward(xd)
    got = {"y": y, **layer.backward(xd, dyd)}
    want = reference(layer, x.astype(np.float64), layer.positions.cpu().numpy(), w_qkv, w_out, gamma, beta, dy,
                     [t // batch] * batch)
    errs = {n: off(got[n].double().cpu().numpy().reshape(want[n].shape), want[n]) for n in want}
    say(" ".join(f"{n}={e:.2e}" for n, e in errs.items()))
    assert all(e < 0.02 for e in errs.values()), errs


def test_sharding_does_not_change_the_branch(gpu_lib):
    """The same cells in another shard order: each row of the output is the same
    sum in another order."""
    from halo_sharded_conv_amd.attention_layer import ShardedAttention
    rng = np.random.default_rng(1)
    spatial, c = (6, 10), 32
    w_qkv, w_out = rng.normal(size=(4 * 16 + 2 * 2 * 16, c)) / 6, rng.normal(size=(c, 64)) / 8
    x = np.float32(rng.normal(size=(*spatial, c)))
    outs = []
    for shards in (((6,), (10,)), ((2, 4), (7, 3))):
        layer = ShardedAttention(spatial, shards, c, 4, 2, 16)
        layer.set_weights(w_qkv, w_out)
        pos = layer.positions.cpu().numpy()
        y = layer.forward(torch.from_numpy(x[pos[:, 0], pos[:, 1]]).cuda()).cpu().numpy()
        whole = np.empty_like(x)
        whole[pos[:, 0], pos[:, 1]] = y
        outs.append(whole)
    assert off(outs[1], outs[0]) < 0.01


def test_refusals(gpu_lib):
    from halo_sharded_conv_amd.attention_layer import ShardedAttention
    with pytest.raises(gpu_lib.ShardConvError):
        ShardedAttention((6, 10), ((3, 3), (10,)), 32, 4, 2, 16, batch=2)
    with pytest.raises(gpu_lib.ShardConvError):
        ShardedAttention((6, 10), ((6,), (10,)), 32, 4, 3, 16)


def test_steps_on_a_stream_of_their_own(gpu_lib):
    """Constructor, weights and the first backward while the current stream is
    busy, every step on another stream: the bits of a run on one stream."""
    from halo_sharded_conv_amd.attention_layer import ShardedAttention
    rng = np.random.default_rng(2)
    w_qkv, w_out = rng.normal(size=(4 * 16 + 2 * 2 * 16, 32)) / 6, rng.normal(size=(32, 64)) / 8
    gamma, beta = 1 + 0.2 * rng.normal(size=32), 0.2 * rng.normal(size=32)
    x = torch.from_numpy(np.float32(rng.normal(size=(60, 32)))).cuda()
    dy = torch.from_numpy(rng.normal(size=(60, 32))).bfloat16().cuda()
    busy = torch.empty(1 << 29, device="cuda")
    torch.cuda.synchronize()

    def steps(stream):
        for _ in range(20):
            busy.fill_(1.0)
        layer = ShardedAttention((6, 10), ((2, 4), (10,)), 32, 4, 2, 16)
        layer.set_weights(w_qkv, w_out, gamma, beta)
        layer.forward(x, stream)
        for _ in range(20):
            busy.fill_(2.0)
        r = layer.backward(x, dy, stream)
        torch.cuda.synchronize()
        return {"y": layer.y, **r}

    want, got = steps(None), steps(torch.cuda.Stream())
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("spatial,shards", [((9, 7), ((5, 4), (4, 3))), ((5, 7, 9), ((2, 3), (7,), (4, 5)))])
def test_odd_shards(gpu_lib, spatial, shards):
    """Shards that start after an odd number of cells."""
    from halo_sharded_conv_amd.attention_layer import ShardedAttention
    rng = np.random.default_rng(3)
    c = 40
    layer = ShardedAttention(spatial, shards, c, 3, 1, 16)
    t = layer.tokens
    pos = layer.positions.cpu().numpy()
    assert sorted(map(tuple, pos)) == sorted(np.ndindex(*spatial))
    x = np.float32(rng.normal(size=(t, c)) + 0.3)
    w_qkv = bf16(rng.normal(size=(layer.joint_width, c)) / np.sqrt(c))
    w_out = bf16(rng.normal(size=(c, layer.width)) / np.sqrt(layer.width))
    gamma, beta = np.float32(1 + 0.2 * rng.normal(size=c)), np.float32(0.2 * rng.normal(size=c))
    dy = bf16(rng.normal(size=(t, c)))
    layer.set_weights(w_qkv, w_out, gamma, beta)
    xd, dyd = torch.from_numpy(x).cuda(), torch.from_numpy(dy).bfloat16().cuda()
    got = {"y": layer.forward(xd), **layer.backward(xd, dyd)}
    want = reference(layer, x.astype(np.float64), pos, w_qkv, w_out, gamma, beta, dy, [t])
    errs = {n: off(got[n].double().cpu().numpy().reshape(want[n].shape), want[n]) for n in want}
    assert all(e < 0.02 for e in errs.values()), errs


@pytest.mark.parametrize("eager_backward", [True, False])
def test_captured_branch(gpu_lib, eager_backward):
    """Forward and backward in one graph, its buffers allocated before or inside
    the capture: every replay gives the eager bits, with weights set in between."""
    from halo_sharded_conv_amd.attention_layer import ShardedAttention
    rng = np.random.default_rng(4)
    weights = [(rng.normal(size=(4 * 16 + 2 * 2 * 16, 32)) / 6, rng.normal(size=(32, 64)) / 8,
                1 + 0.2 * rng.normal(size=32), 0.2 * rng.normal(size=32)) for _ in range(2)]
    x = torch.from_numpy(np.float32(rng.normal(size=(60, 32)))).cuda()
    dy = torch.from_numpy(rng.normal(size=(60, 32))).bfloat16().cuda()

    def make():
        layer = ShardedAttention((6, 10), ((2, 4), (10,)), 32, 4, 2, 16)
        layer.set_weights(*weights[0])
        return layer

    layer, eager = make(), make()
    layer.forward(x)
    if eager_backward:
        layer.backward(x, dy)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(x)
        grads = layer.backward(x, dy)
    for i in range(4):
        for one in (layer, eager):
            one.set_weights(*weights[i % 2])
        want = {"y": eager.forward(x), **eager.backward(x, dy)}
        for t in (layer.y, *grads.values()):
            t.fill_(float(i))
        g.replay()
        torch.cuda.synchronize()
        for n, t in {"y": layer.y, **grads}.items():
            assert torch.equal(t, want[n]), (i, n)
