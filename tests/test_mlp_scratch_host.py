"""Layers of the MLP branch with 8-bit products on one set of scratch, without a GPU."""
import numpy as np
import pytest
import torch

import halo_sharded_conv_amd as hsc
from test_mlp_layer_host import events, make, names  # noqa: F401


@pytest.mark.parametrize("kept", [("bf16", "bf16"), ("mx8", "bf16"), ("bf16", "mx8")])
def test_eight_bit_products_share_scratch(events, kept):  # noqa: F811
    """No backward pass reads their buffers, whatever `kept` says."""
    a = make(products="mx8", kept=kept[0])
    b = make(products="mx8", kept=kept[1], scratch=a)
    for n in ("total", "normed8", "h", "h8", "y"):
        assert getattr(a, n) is getattr(b, n)
    assert b.w_up is not a.w_up and b.w_down is not a.w_down and b.ws is not a.ws
    events.clear()
    b.forward(a.y)
    assert names(events) == ["st_rmsnorm", "st_linear", "st_mx8_store", "st_linear"]


def test_scratch_that_stays_refused(events):  # noqa: F811
    eight = make(products="mx8")
    for other in (dict(), dict(kept="mx8"), dict(products="mx8", hidden=96), dict(products="mx8", channels=64)):
        with pytest.raises(hsc.ShardConvError) as e:
            make(scratch=eight, **other)
        assert e.value.status == 2
    with pytest.raises(hsc.ShardConvError) as e:
        make(scratch=make())
    assert e.value.status == 4
