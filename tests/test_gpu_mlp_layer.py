"""The MLP branch (RMS norm with the branch's addition, two products, and their
gradients) against its fp64 definition, alone, behind the attention branch, on
streams and in graphs.

Tolerance: every bf16 rounding on the way (the normed cells, the hidden values
and their gradients, p: at most 6 in a row) is off by 2^-9 of its value in the
mean square, every e4m3 rounding by 2^-5 (half of the largest, 2^-4); independent
errors add in squares and each step's gain is about one: sqrt(6) 2^-9 = 0.5%,
held to 2% of the norm, and with three 8-bit tensors in a row sqrt(3) 2^-5 = 5.4%,
held to 10%.

ReLU's slope jumps at zero, so the sign of a pre-activation that the rounding of
the normed cells turns over counts whole.  p is normal with deviation s, its
error e has a deviation of about 2^-9 s: a share E|e| / (s sqrt(2 pi)) = 0.8 * 2^-9
* 0.4 = 6.2e-4 of the values turns over, and half of them have a gradient, so the
gradients behind them are off by sqrt(6.2e-4 / 0.5) = 3.5% of the norm.  In the case
below (192 cells, 96 wide) that is 11 values; 3 deviations more, 21, are 4.8%, with
the 2% above 5.2%: held to 6%.
"""
import numpy as np
import pytest
import torch

from helpers import say
from oracle import mlp

pytestmark = pytest.mark.gpu


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().double().numpy()


def weights(c, h, seed=0):
    rng = np.random.default_rng(seed)
    return {"w_up": bf16(rng.normal(size=(h, c)) / np.sqrt(c)), "w_down": bf16(rng.normal(size=(c, h)) / np.sqrt(h)),
            "b_up": np.float32(0.2 * rng.normal(size=h)), "b_down": np.float32(0.2 * rng.normal(size=c)),
            "gamma": np.float32(1 + 0.2 * rng.normal(size=c))}


def reference(x, branch, w, act, dy, eps):
    s = x + branch
    n, _ = mlp.rms_norm(s, w["gamma"], eps)
    h, pre = mlp.linear(n, w["w_up"], w["b_up"], act)
    y, _ = mlp.linear(h, w["w_down"], w["b_down"], "none", s)
    dh, dw_down, db_down = mlp.linear_backward(h, w["w_down"], dy)
    dn, dw_up, db_up = mlp.linear_backward(n, w["w_up"], dh, act, pre)
    dx, dg = mlp.rms_norm_backward(s, dn, dy, w["gamma"], eps=eps)
    return {"y": y, "dx": dx, "dw_up": dw_up, "db_up": db_up, "dw_down": dw_down, "db_down": db_down, "dgamma": dg}


def off(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("spatial,shards,batch,channels,hidden,act", [
    ((9, 14), ((4, 5), (14,)), 1, 32, 128, "gelu"),
    ((4, 6, 10), ((4,), (6,), (7, 3)), 1, 50, 130, "silu"),      # rows off the 16-byte grid
    ((8, 8), ((8,), (8,)), 3, 72, 96, "relu"),
    ((40, 30), ((40,), (30,)), 1, 256, 1024, "gelu"),
    ((1, 1), ((1,), (1,)), 1, 64, 256, "gelu"),                  # one cell
])
@pytest.mark.parametrize("kept", ["bf16", "mx8"])
def test_branch(gpu_lib, spatial, shards, batch, channels, hidden, act, kept):
    from halo_sharded_conv_amd.mlp_layer import ShardedMLP
    say(f"MLP branch {spatial} {shards} C={channels} hidden {hidden} {act} {kept}")
    layer = ShardedMLP(spatial, shards, channels, hidden, act, kept=kept, batch=batch)
    rng = np.random.default_rng(1)
    t = layer.tokens
    assert t == batch * int(np.prod(spatial)) and len(layer.parts(layer.total)) == int(np.prod([len(s) for s in shards]))
    x, branch = np.float32(rng.normal(size=(t, channels))), bf16(rng.normal(size=(t, channels)))
    dy = np.float32(rng.normal(size=(t, channels)))
    w = weights(channels, hidden)
    layer.set_weights(**w)
    xd, bd, dyd = torch.from_numpy(x).cuda(), torch.from_numpy(branch).bfloat16().cuda(), torch.from_numpy(dy).cuda()
    y = layer.forward(xd, bd)
    got = {"y": y, **layer.backward(dyd)}
    want = reference(x.astype(np.float64), branch, w, act, dy.astype(np.float64), layer.eps)
    errs = {n: off(got[n].double().cpu().numpy(), want[n]) for n in want}
    say(" ".join(f"{n}={e:.2e}" for n, e in errs.items()))
    assert errs["y"] < 0.02 and errs["db_down"] < 1e-5
    assert all(e < (0.1 if kept == "mx8" else 0.06 if act == "relu" else 0.02) for e in errs.values()), errs


def test_eight_bit_products(gpu_lib):
    from halo_sharded_conv_amd.mlp_layer import ShardedMLP
    layer = ShardedMLP((20, 30), ((8, 12), (30,)), 96, 384, products="mx8")
    rng = np.random.default_rng(2)
    x = np.float32(rng.normal(size=(600, 96)))
    w = weights(96, 384)
    layer.set_weights(**w)
    y = layer.forward(torch.from_numpy(x).cuda())
    want = reference(x.astype(np.float64), 0.0, w, "gelu", np.zeros((600, 96)), layer.eps)["y"]
    # four 8-bit roundings (two weights, two inputs) on the branch, half of the output
    assert off(y.double().cpu().numpy(), want) < 0.1
    with pytest.raises(gpu_lib.ShardConvError):
        layer.backward(torch.zeros(600, 96, device="cuda"))


def test_layers_share_scratch(gpu_lib):
    """Two 8-bit layers on one set of scratch give what two of their own do."""
    from halo_sharded_conv_amd.mlp_layer import ShardedMLP
    args = ((12, 10), ((5, 7), (10,)), 64, 160)
    rng = np.random.default_rng(3)
    x = torch.from_numpy(np.float32(rng.normal(size=(120, 64)))).cuda()
    dy = torch.from_numpy(np.float32(rng.normal(size=(120, 64)))).cuda()
    outs = []
    for shared in (False, True):
        a = ShardedMLP(*args, kept="mx8")
        b = ShardedMLP(*args, kept="mx8", scratch=a if shared else None)
        a.set_weights(**weights(64, 160, 5))
        b.set_weights(**weights(64, 160, 6))
        ya = a.forward(x).clone()
        yb = b.forward(ya).clone()
        gb = {n: v.clone() for n, v in b.backward(dy).items()}
        ga = {n: v.clone() for n, v in a.backward(gb["dx"]).items()}
        outs.append([yb, *gb.values(), *ga.values()])
        if shared:                               # without the copies: y is the next x, dx the dy before
            b.forward(a.forward(x))
            assert torch.equal(b.y, yb)
            again = a.backward(b.backward(dy)["dx"])
            assert all(torch.equal(again[n], ga[n]) for n in ga)
    assert all(torch.equal(p, q) for p, q in zip(*outs))
    with pytest.raises(gpu_lib.ShardConvError):
        ShardedMLP((12, 10), ((5, 7), (10,)), 64, 128, kept="mx8", scratch=a)


def test_block_of_both_branches(gpu_lib):
    """attention, then the MLP on x + attention: forward and backward together, as
    a transformer block runs them, against the MLP's definition on the attention's
    own output."""
    from halo_sharded_conv_amd.attention_layer import ShardedAttention
    from halo_sharded_conv_amd.mlp_layer import ShardedMLP
    spatial, shards, c = (10, 12), ((4, 6), (12,)), 64
    rng = np.random.default_rng(4)
    att = ShardedAttention(spatial, shards, c, 4, 2, 16)
    att.set_weights(rng.normal(size=(att.joint_width, c)) / 8, rng.normal(size=(c, att.width)) / 8)
    layer = ShardedMLP(spatial, shards, c, 256)
    w = weights(c, 256)
    layer.set_weights(**w)
    x = torch.from_numpy(np.float32(rng.normal(size=(120, c)))).cuda()
    dy = torch.from_numpy(np.float32(rng.normal(size=(120, c)))).cuda()
    branch = att.forward(x)
    y = layer.forward(x, branch)
    g = layer.backward(dy)
    da = att.backward(x, g["dx"].bfloat16())
    want = reference(x.double().cpu().numpy(), branch.double().cpu().numpy(), w, "gelu", dy.double().cpu().numpy(), layer.eps)
    assert off(y.double().cpu().numpy(), want["y"]) < 0.02 and off(g["dx"].double().cpu().numpy(), want["dx"]) < 0.02
    assert bool(torch.isfinite(da["dx"]).all())


@pytest.mark.parametrize("kept", ["bf16", "mx8"])
def test_steps_on_a_stream_of_their_own_and_captured(gpu_lib, kept):
    """The bits of a run on one stream: on another while the current one is busy, and
    replayed from a graph with eager work in between."""
    from halo_sharded_conv_amd.mlp_layer import ShardedMLP
    args = ((30, 20), ((30,), (20,)), 128, 520)
    rng = np.random.default_rng(5)
    x = torch.from_numpy(np.float32(rng.normal(size=(600, 128)))).cuda()
    dy = torch.from_numpy(np.float32(rng.normal(size=(600, 128)))).cuda()
    layer = ShardedMLP(*args, kept=kept)
    layer.set_weights(**weights(128, 520))
    want = [layer.forward(x).clone(), *(v.clone() for v in layer.backward(dy).values())]
    other = ShardedMLP(*args, kept=kept)
    busy = torch.empty(1 << 28, device="cuda")
    for _ in range(20):
        busy.add_(1.0)
    other.set_weights(**weights(128, 520))
    side = torch.cuda.Stream()
    for _ in range(20):
        busy.add_(1.0)
    y = other.forward(x, stream=side)
    g = other.backward(dy, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, [y, *g.values()]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.forward(x)
        other.backward(dy)
    for i in range(3):
        for v in (other.y, *other.grads.values()):
            v.zero_()
        layer.forward(x)                                  # eager work of another layer between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [other.y, *(other.grads[n] for n in g)])), f"replay {i}"


def test_two_calls_at_once(gpu_lib):
    """Calls on two streams with a workspace each, several times over."""
    m, k, n = 700, 512, 264
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.normal(size=(m, k))).bfloat16().cuda()
    ws_bytes = gpu_lib.st_linear_workspace_bytes(m, k, n, "bf16", backward=True)
    w = [torch.from_numpy(rng.normal(size=(n, k)) / 22).bfloat16().cuda() for _ in range(2)]
    dy = torch.from_numpy(rng.normal(size=(m, n))).bfloat16().cuda()
    want = []
    for i in range(2):
        dx, dw, db = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
        gpu_lib.st_linear_backward(x, w[i], dy, dx, dw, db, workspace=torch.empty(ws_bytes, dtype=torch.uint8, device="cuda"))
        want.append((dx, dw, db))
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(ws_bytes, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [[torch.empty_like(v) for v in want[i]] for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            gpu_lib.st_linear_backward(x, w[i], dy, *outs[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
