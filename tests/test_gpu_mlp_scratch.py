"""Layers of the MLP branch with 8-bit products that share scratch."""
import numpy as np
import pytest
import torch

from test_gpu_mlp_layer import weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("args", [((12, 10), ((5, 7), (10,)), 64, 160), ((1, 1), ((1,), (1,)), 50, 130), ((30, 40), ((10, 20), (40,)), 256, 520)])
def test_eight_bit_layers_share_scratch(gpu_lib, args):
    """Two in a row, the second's stream the first's output where it lies: the bits of
    two layers with buffers of their own, call after call and replayed from a graph."""
    from halo_sharded_conv_amd.mlp_layer import ShardedMLP
    channels, hidden = args[2:]
    rng = np.random.default_rng(21)
    own = [ShardedMLP(*args, products="mx8") for _ in range(2)]
    a = ShardedMLP(*args, products="mx8")
    both = [a, ShardedMLP(*args, products="mx8", scratch=a)]
    for layers in (own, both):
        for i, layer in enumerate(layers):
            layer.set_weights(**weights(channels, hidden, 30 + i))
    x = torch.from_numpy(np.float32(rng.normal(size=(a.tokens, channels)))).cuda()
    want = own[1].forward(own[0].forward(x)).clone()
    assert bool(torch.isfinite(want).all()) and both[0].y is both[1].y
    for _ in range(2):
        assert torch.equal(both[1].forward(both[0].forward(x)), want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both[1].forward(both[0].forward(x))
    for i in range(3):
        both[1].y.zero_()
        assert torch.equal(own[1].forward(own[0].forward(x)), want)       # eager work between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(both[1].y, want), f"replay {i}"
